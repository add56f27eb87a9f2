"""The forms that allocate, given a stream that is not torch's current one (needs a GPU):
they take no memory that the current stream still uses, leave none to it that they still use,
and read back what their own stream has written."""
import dataclasses

import pytest
import torch

from logprob_drift_scoring_gb300 import binding as B
from logprob_drift_scoring_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"


def case(name):
    """The form as a function of its stream."""
    g = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    rows, vocab = 300, 5003
    x, y = rand(rows, vocab).bfloat16(), rand(rows, vocab).bfloat16()
    ids = torch.randint(0, vocab, (rows,), generator=g, device=DEV, dtype=torch.int32)
    act, u = torch.ones(rows, dtype=torch.uint8, device=DEV), torch.rand(rows, generator=g, device=DEV)
    logps, small = [rand(rows) for _ in range(4)], rand(rows) * 0.01
    if name in ("micro_matmul", "block_matmul"):
        quantize = B.micro_quantize if name == "micro_matmul" else B.block_quantize
        a, b = quantize(rand(64, 20000).bfloat16()), quantize(rand(300, 20000).bfloat16())  # (a split k axis)
        return lambda s: getattr(B, name)(a, b, torch.float32, stream=s)
    if name == "score_fused":
        h = W.head(rows, 256, 1000)
        return lambda s: B.score_fused(h.hidden_train, h.hidden_rollout, h.weight, h.token_ids, h.action_mask, stream=s)
    if name == "score_sharded_topology":
        cuts = [(0, 2000), (2000, vocab)]
        xs, ys = ([t[:, a:b].contiguous() for a, b in cuts] for t in (x, y))
        return lambda s: B.score_sharded_topology(xs, ys, cuts, ids, act, 0, stream=s)
    if name in ("attn_merge", "attn_merge_order_drift"):
        a = W.attn_partials(300, 3, 128, 5, seed=3, device=DEV)
        return lambda s: getattr(B, name)(a.out_parts, a.lse_parts, [4, 3, 2, 1, 0], stream=s)
    return {
        "sample": lambda s: B.sample(x, u, stream=s),
        "filter_mask": lambda s: B.filter_mask(x, None, ids, act, s),
        "micro_quantize": lambda s: B.micro_quantize(x, stream=s),
        "block_quantize": lambda s: B.block_quantize(x, stream=s),
        "controls_apply": lambda s: B.controls_apply(x, B.Controls(scale=u), stream=s),
        "score": lambda s: B.score(x, y, ids, act, stream=s),
        "score_controlled": lambda s: B.score_controlled(x, y, ids, act, stream=s),
        "logp_drift_summary": lambda s: B.logp_drift_summary(*logps, act, stream=s),
        "drift_metrics_from_dlogp": lambda s: B.drift_metrics_from_dlogp(small, act, stream=s),
    }[name]


NAMES = ["sample", "filter_mask", "micro_quantize", "micro_matmul", "block_quantize", "block_matmul", "controls_apply", "score",
         "score_controlled", "score_fused", "score_sharded_topology", "attn_merge", "attn_merge_order_drift", "logp_drift_summary",
         "drift_metrics_from_dlogp"]


def parts(res):
    """The tensors and the other values of a result."""
    if isinstance(res, torch.Tensor):
        return [res], []
    if isinstance(res, dict):
        return [], [res]
    if dataclasses.is_dataclass(res):
        res = [getattr(res, f.name) for f in dataclasses.fields(res)]
    if isinstance(res, (list, tuple)):
        both = [parts(r) for r in res]
        return sum((t for t, _ in both), []), sum((v for _, v in both), [])
    return [], [res]


def busy(big):
    """Some 20 ms of work on the current stream."""
    for _ in range(40):
        big.mul_(1.0)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_uses(name, handle):
    form = case(name)
    want, other = parts(form(None))
    big = torch.ones(1 << 29, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sizes = [t.untyped_storage().nbytes() for t in want] + [B.METRICS_BYTES, B.MERGE_DRIFT_BYTES, B.LOGP_DRIFT_BYTES]
    old = [torch.full((max(n, 1),), 7, dtype=torch.uint8, device=DEV) for n in sizes]
    copies = [torch.empty_like(t) for t in old]
    torch.cuda.synchronize()
    busy(big)
    for c, t in zip(copies, old):
        c.copy_(t)
    del t, old  # (torch may give their memory to whatever the current stream does next)
    got, values = parts(form(side.cuda_stream if handle else side))
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies)
    assert values == other and len(got) == len(want)
    assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_a_busy_stream(name):
    """The form's work waits on its stream; what the current stream allocates meanwhile is its own."""
    form = case(name)
    want, other = parts(form(None))
    big = torch.ones(1 << 29, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        busy(big)
    got, values = parts(form(side))
    room = [torch.full((1 << k,), 0xFF, dtype=torch.uint8, device=DEV) for k in range(9, 26)]
    torch.cuda.synchronize()
    assert values == other and all(bool((r == 0xFF).all()) for r in room)
    assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(got, want))
