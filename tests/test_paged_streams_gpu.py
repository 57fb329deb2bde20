"""What a plan holds outlives the calls that read it, on whichever stream they run."""

import pytest
import torch

from gpu_util import fa_mod
from paged_util import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("anew", [False, True])
@pytest.mark.parametrize("chunk", [1, 40])
def test_a_table_of_another_stream_is_kept_while_it_is_read(anew, chunk):
    # The table belongs to the current stream, the plan and all its calls to another, which is behind. Dropped, or
    # replaced by laying the plan out anew, the table's memory is not handed out again until the calls are done.
    fa = fa_mod()
    b = Batch([(chunk, 300), (1, 100)], 8, 2, 128, 16, seed=51)
    wide = torch.zeros(2, 3_500_000, dtype=torch.int32)
    wide[:, :b.table.shape[1]] = b.table
    s = torch.cuda.Stream()
    tables = [wide.cuda() for _ in range(2 if anew else 1)]
    b.dev["table"] = tables[0]
    torch.cuda.synchronize()
    fa.forward_paged(b.dev["q"], b.kc, b.vc, b.plan(fa, stream=s), stream=s)  # loads the code, and memory for s to have
    torch.cuda.synchronize()
    del tables[0], b.dev["table"]
    table = b.dev["table"] = wide.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)  # about a fifth of a second
    plan = b.plan(fa, stream=s)
    o, lse = fa.forward_paged(b.dev["q"], b.kc, b.vc, plan, stream=s)
    address = table.data_ptr()
    del table
    del b.dev["table"]
    if anew:
        b.dev["table"] = tables[0]
        b.plan(fa, plan=plan, stream=s)
    else:
        del plan
    busy = not s.query()
    taken = torch.empty(wide.shape, dtype=torch.int32, device="cuda").data_ptr() == address
    fa.check(stream=s)
    b.check(o, lse)
    assert busy and not taken


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("lens", [[(1, 3000)] * 20, [(160, 2000), (1, 900), (40, 500)], [(1, 9000)]])
def test_calls_at_once_with_a_plan_each(lens, captured):
    # Two streams, each with batches of its own plan under way at the same time, eager or as captured graphs.
    fa = fa_mod()
    batches = [Batch(lens, 8, 2, d, 32, seed=52 + d) for d in (64, 128)]
    streams = [torch.cuda.Stream() for _ in batches]
    plans = [b.plan(fa) for b in batches]
    outs = [fa.forward_paged(b.dev["q"], b.kc, b.vc, p) for b, p in zip(batches, plans)]
    fa.check()
    want = [(o.clone(), lse.clone()) for o, lse in outs]

    def call(i, stream=None):
        b = batches[i]
        b.plan(fa, plan=plans[i], stream=stream)
        fa.forward_paged(b.dev["q"], b.kc, b.vc, plans[i], out=outs[i][0], lse=outs[i][1], stream=stream)

    graphs = []
    if captured:
        for i in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                for _ in range(3):
                    call(i)
    for o, lse in outs:
        o.zero_()
        lse.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            if captured:
                with torch.cuda.stream(s):
                    graphs[i].replay()
            else:
                call(i, s)
    for s in streams:
        fa.check(stream=s)
    for b, (o, lse), (wo, wl) in zip(batches, outs, want):
        b.check(o, lse)
        assert torch.equal(o, wo) and torch.equal(lse, wl)
