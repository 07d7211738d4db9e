"""The norm, router and expert calls as they are used: together, in HIP graphs,
on other streams, with padded batches, rows that hold no numbers, and calls at
once; and the example.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_04_amd as fb
from tests.gpu_util import DEV, require_gpu
from tests.layer_util import EXPERT_ARGS, expert_case, expert_dev

pytestmark = pytest.mark.gpu


def setup_module(module):
    require_gpu()


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def block(x, r, weight, router, w):
    """norm -> router -> experts; every intermediate result."""
    q, s, h, rstd, y = fb.rms_norm_quantize(x, weight, residual=r, return_y=True)
    logits = (y.float()[:, None] * router[None]).sum(2)           # (elementwise and one reduction over a row)
    ids, wt = fb.moe_route(logits, 2)
    out = fb.moe_experts(q, s, ids, wt, *w)
    dl = fb.moe_route_backward(logits, ids, wt)
    dx, dw = fb.rms_norm_backward(out, h, rstd, weight, dh=r)
    return q, s, h, rstd, y, ids, wt, out, dl, dx, dw


@pytest.mark.parametrize("tokens", [1, 20, 70])
def test_captured_chain_follows_its_inputs(tokens):
    w = expert_dev(expert_case(tokens, 256, 128, 6, 2, seed=1))[4:]
    gen = torch.Generator(device=DEV).manual_seed(2)
    rand = lambda *n: torch.randn(*n, generator=gen, device=DEV)  # noqa: E731
    x, r = rand(tokens, 256).bfloat16(), rand(tokens, 256).bfloat16()
    weight, router = 1 + 0.1 * rand(256), rand(6, 256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, r, weight, router, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(x, r, weight, router, w)
    for k in range(4):
        x.copy_(rand(tokens, 256))
        r.copy_(rand(tokens, 256))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = block(x, r, weight, router, w)
        torch.cuda.synchronize()
        assert same(kept, want), k


@pytest.mark.parametrize("T,E", [(2, 8), (40, 4)])
def test_two_graphs_share_a_workspace(T, E):
    cases = [expert_dev(expert_case(T, 256, 256, E, 2, seed=k)) for k in range(2)]
    ws = torch.empty(fb.moe_experts_workspace_bytes(T, 256, 256, E, 2), dtype=torch.uint8, device=DEV)
    want = [fb.moe_experts(*c) for c in cases]
    rows = [torch.randn(50, 256, device=DEV).bfloat16() for _ in range(2)]
    nws = torch.empty(fb.rms_norm_backward_workspace_bytes(50, 256), dtype=torch.uint8, device=DEV)
    rstd, weight = torch.rand(50, device=DEV), torch.rand(256, device=DEV)
    back = [fb.rms_norm_backward(x, x, rstd, weight) for x in rows]
    torch.cuda.synchronize()
    graphs, got = [], []
    for c, x in zip(cases, rows):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append((fb.moe_experts(*c, workspace=ws), *fb.rms_norm_backward(x, x, rstd, weight, workspace=nws)))
    for k in (0, 1, 1, 0, 0, 1):
        for t in got[k]:
            t.zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        assert same(got[k], (want[k], *back[k])), k


def test_calls_on_two_streams_at_once():
    cases = [expert_dev(expert_case(T, 256, 256, 8, 2, seed=T)) for T in (3, 64)]
    x = torch.randn(700, 1024, device=DEV).bfloat16()
    weight, rstd = torch.rand(1024, device=DEV), torch.rand(700, device=DEV)
    logits = torch.randn(3000, 64, device=DEV)

    def all_of(c):
        return (fb.moe_experts(*c), *fb.rms_norm_quantize(x, weight), *fb.rms_norm_backward(x, x, rstd, weight),
                *fb.moe_route(logits, 6))
    want = [all_of(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        now = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                now.append(all_of(c))
        got.append(now)
    torch.cuda.synchronize()
    for now in got:
        for a, b in zip(now, want):
            assert same(a, b)


@pytest.mark.parametrize("T,E,topk", [(9, 16, 2), (40, 4, 2), (100, 3, 1)])
def test_rows_without_numbers_stay_alone(T, E, topk):
    # padded tokens of NaN codes and scales give 0; a token of NaN gives NaN and leaves the others' bits alone;
    # experts that no token has may hold anything
    w = expert_case(T, 256, 128, E + 1, topk, seed=5)
    w["ids"][w["ids"] == E] = 0
    w["ids"][T // 2:T // 2 + 3] = -1
    want = fb.moe_experts(*expert_dev(w))
    w["x"][T // 2:T // 2 + 3] = 0x7F
    w["sx"][:, T // 2:T // 2 + 3] = np.nan
    w["weights"][T // 2:T // 2 + 3] = np.nan
    for n in ("w13", "w2"):
        w[n][E] = 0x7F
        w["s" + n[1:]][E] = np.nan
    got = fb.moe_experts(*expert_dev(w))
    assert same([got], [want]) and (got[T // 2:T // 2 + 3] == 0).all()
    w["x"][0, 77] = 0xFF
    got = fb.moe_experts(*expert_dev(w))
    assert torch.isnan(got[0]).all() and same([got[1:]], [want[1:]])


def test_large_experts_pass_32_bits():
    # weights of 5 x 2^29 codes: the last experts' offsets pass 2^31
    H, I, E = 16384, 16384, 5
    w13 = torch.zeros(E, 2 * I, H, dtype=torch.uint8, device=DEV)
    w2 = torch.zeros(E, H, I, dtype=torch.uint8, device=DEV)
    one = 0x38                                            # E4M3 of 1
    x = torch.full((1, H), one, dtype=torch.uint8, device=DEV)
    w13[E - 1, :I, :128] = one                            # gates of 128
    w13[E - 1, 2 * I - 3, H - 1] = one                    # u = 1 in one column
    w2[E - 1, H - 5, I - 3] = one
    ones = lambda *n: torch.ones(*n, device=DEV)  # noqa: E731
    for ids in ([E - 1], [E - 1, 0], [2, 3, E - 1, 0, 1]):
        got = fb.moe_experts(x, ones(H // 128, 1), torch.tensor([ids], dtype=torch.int32, device=DEV), ones(1, len(ids)),
                             w13, ones(E, 2 * I // 128, H // 128), w2, ones(E, H // 128, I // 128),
                             out_dtype=torch.float32)
        assert got[0, H - 5] == 128 and got.sum() == 128
    del w13, w2
    torch.cuda.empty_cache()


def test_large_rows_pass_32_bits():
    # 300000 rows of 8192: element offsets pass 2^31
    m, k = 300000, 8192
    x = torch.ones(m, k, dtype=torch.bfloat16, device=DEV)
    x[m - 1, ::2] = -3.0
    weight = torch.ones(k, device=DEV)
    q, s, _, rstd = fb.rms_norm_quantize(x, weight, 2.0 ** -100)
    q1, s1, _, rstd1 = fb.rms_norm_quantize(x[m - 2:].contiguous(), weight, 2.0 ** -100)
    assert same([q[m - 2:], rstd[m - 2:]], [q1, rstd1]) and torch.equal(s[:, m - 2:], s1)
    del q, s
    dx, _ = fb.rms_norm_backward(x, x, rstd, weight)
    assert same([dx[m - 2:]], [fb.rms_norm_backward(x[m - 2:].contiguous(), x[m - 2:].contiguous(), rstd1, weight)[0]])
    del x, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("pow2", [False, True])
def test_norm_feeds_the_gemms(pow2):
    # codes and scales go into the dense GEMM as they are: its product of their values, within the GEMMs' tolerance
    from oracle import gemm
    from tests.gpu_util import ABS_RMS, REL, codes_host
    gen = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(37, 1024, generator=gen, device=DEV).bfloat16()
    w = (0.02 * torch.randn(256, 1024, generator=gen, device=DEV)).bfloat16()
    q, s, _, _ = fb.rms_norm_quantize(x, torch.rand(1024, generator=gen, device=DEV), pow2=pow2)
    wq, ws = fb.quantize_128x128(w, pow2=pow2)
    got = fb.gemm(q, s, wq, ws, out_dtype=torch.float32, pow2_scales=pow2).cpu().numpy().astype(np.float64)
    ref = gemm.gemm_f64(codes_host(q), s.cpu().numpy(), codes_host(wq), ws.cpu().numpy())
    assert np.all(np.abs(got - ref) <= REL * np.abs(ref) + ABS_RMS * np.sqrt(np.mean(ref ** 2)))


def test_norm_without_its_optional_outputs():
    # through the C ABI: rstd and y NULL leave the others as they are
    from fp8_block_scaled_04_amd import fp8bs
    x, w = torch.randn(9, 384, device=DEV).bfloat16(), torch.rand(384, device=DEV)
    want = fb.rms_norm_quantize(x, w)
    q, s = torch.empty_like(want[0]), torch.empty_like(want[1])
    status = fp8bs._norm(x.data_ptr(), None, w.data_ptr(), 1, 1e-6, 9, 384, None, None, q.data_ptr(), s.data_ptr(), None,
                         0, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0 and same([q, s], want[:2])


def test_gradients_accumulate_over_parts():
    # two halves of a batch into one dweight: the sum of theirs
    x = torch.randn(60, 256, device=DEV).bfloat16()
    w, rstd = torch.rand(256, device=DEV), torch.rand(60, device=DEV)
    parts = [fb.rms_norm_backward(x[i:i + 30], x[i:i + 30], rstd[i:i + 30], w) for i in (0, 30)]
    acc = torch.zeros(256, device=DEV)
    dx = [fb.rms_norm_backward(x[i:i + 30], x[i:i + 30], rstd[i:i + 30], w, dweight=acc, accumulate=True)[0] for i in (0, 30)]
    assert same(dx, [p[0] for p in parts]) and torch.equal(acc, parts[0][1] + parts[1][1])


def test_arguments_keep_their_values():
    w = expert_dev(expert_case(5, 256, 128, 4, 2, seed=3))
    before = [t.clone() for t in w]
    fb.moe_experts(*w)
    assert same(w, before) and len(w) == len(EXPERT_ARGS)


# The experts' products take E4M3 activations and weights, each within 2^-4 (relative) of its value, 0.026 root mean
# square (2^-4 / sqrt 6): out's error is about 0.026 sqrt 2 through the first product (twice, gate and up), 0.026 from
# w2: 0.058 in all; BF16 sums and outputs 2^-9.  0.15 covers this two and a half times; a wrong expert or row is off by 1.
def test_example_decodes():
    from examples import moe_block
    for tokens in (1, 16, 64):
        _, errors, equal = moe_block.decode(tokens, layers=3, steps=2)
        assert equal and max(errors) < 0.15, (tokens, errors)


# dw: E4M3 operands on both sides, 0.026 sqrt 2 (the activations twice quantized: sqrt 3); dx and dnorm carry dy's
# E4M3 error of 0.026 sqrt 2 and its BF16 rounding; drouter only y's BF16 rounding, through the softmax.
def test_example_gradients():
    from examples import moe_block
    got = moe_block.gradients()
    for name, most in (("dx", 0.1), ("dnorm", 0.1), ("dw", 0.1), ("drouter", 0.02)):
        g, want = got[name]
        assert g.shape == want.shape
        assert float((g.double() - want).norm() / want.norm()) < most, name
