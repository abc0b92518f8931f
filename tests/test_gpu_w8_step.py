"""An 8-bit layer's operators as they are used (examples/mlp_step.py): each stage against its
definition in 64 bits on the values the stage before left; graphs, streams, shared workspaces."""
import os
import sys

import pytest

import heterogeneous_adapters_gb300 as lora

from .test_gpu_w8 import call, check, codes, problem, problems, workspace

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def product(torch, mlp, i, x, codes, scales, adapters):
    """codes W^T by the scales + the deltas of x, fp64, and the size of the sums."""
    w, ws = mlp.weights[i]
    k, n = mlp.dims[i]
    r = mlp.rank
    base = (codes.double() @ w.double().t()) * scales.double()[:, None] * ws.double()
    x = x.double()
    y, size = base.clone(), base.abs()
    pages = lambda d: -(-d // mlp.h)  # noqa: E731
    pre = sum(pages(a) + pages(b) for a, b in mlp.dims[:i])
    for t, a in enumerate(adapters):
        if a < 0:
            continue
        at = int(mlp.pt_off[a]) + r * pre
        rows = mlp.pages[mlp.page_table[at:at + r * (pages(k) + pages(n))].long()].double()
        A = rows[:r * pages(k)].view(pages(k), r, -1).transpose(0, 1).reshape(r, -1)[:, :k]
        B = rows[r * pages(k):].view(pages(n), r, -1).transpose(0, 1).reshape(r, -1)[:, :n]
        y[t] += (x[t] @ A.t()) * 2.0 @ B
        size[t] += (x[t].abs() @ A.abs().t()) * 2.0 @ B.abs()
    return y, size


def check_layer(torch, mlp, x, residual, adapters):
    T, f = x.shape[0], mlp.f
    h = (x.float() + residual.float()).bfloat16()
    assert torch.equal(mlp.residual[:T], h)
    p = h.double() * mlp.norm.double()
    top = p.abs().amax(1, keepdim=True)
    assert torch.equal(mlp.q[:T].double(), torch.round(127 * p / top))
    scale = (top / 127 / torch.sqrt(h.double().square().mean(1, keepdim=True) + 1e-5))[:, 0]
    assert bool(((mlp.qs[:T].double() - scale).abs() <= 2.0 ** -19 * scale).all())
    # the base's product and the sum with the delta round to bf16 (2^-8 each); the delta's own sums are fp32
    near = lambda got, want, size: bool(((got.double() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -7 * size).all())  # noqa: E731
    for i, y in enumerate((mlp.both[:T, :f], mlp.both[:T, f:])):
        assert near(y, *product(torch, mlp, i, mlp.xn[:T], mlp.q[:T], mlp.qs[:T], adapters)), i
    g, u = mlp.both[:T, :f].double(), mlp.both[:T, f:].double()
    y = g * torch.sigmoid(g) * u
    step = mlp.qas[:T].double()[:, None]
    assert bool(((mlp.qa[:T].double() * step - y).abs() <= (0.5 + 2.0 ** -13) * step + 2.0 ** -16 * y.abs()).all())
    assert bool((mlp.qa[:T].abs().amax(1) == 127).all())
    assert near(mlp.out[:T], *product(torch, mlp, 2, mlp.xa[:T], mlp.qa[:T], mlp.qas[:T], adapters))


@pytest.mark.parametrize("h,f,T", [(512, 1408, 1), (512, 1408, 7), (1024, 2816, 40), (256, 768, 300)])
def test_decode_layer(cuda, h, f, T):
    from mlp_step import Mlp
    mlp = Mlp(h, f, rows=T + 3, adapters=5, rank=8)
    g = cuda.Generator(device="cuda").manual_seed(T)
    adapter = cuda.randint(-1, 5, (T,), generator=g, device="cuda").int()
    for _ in range(2):
        x, res = (cuda.randn(T, h, generator=g, device="cuda").bfloat16() for _ in range(2))
        mlp.step(x, res, adapter)
        assert mlp.errors() == 0
        check_layer(cuda, mlp, x, res, adapter.tolist())


def test_prompt_layer(cuda):
    from mlp_step import Mlp
    mlp = Mlp(512, 1408, rows=900, adapters=4, rank=16)
    start, which = [0, 500, 501, 640, 900], [2, -1, 0, 3]
    adapters = [w for w, a, b in zip(which, start, start[1:]) for _ in range(b - a)]
    x, res = (cuda.randn(900, 512, device="cuda").bfloat16() for _ in range(2))
    mlp.step(x, res, None, cuda.tensor(start, device="cuda").int(), cuda.tensor(which, device="cuda").int())
    assert mlp.errors() == 0
    check_layer(cuda, mlp, x, res, adapters)


@pytest.mark.parametrize("T", [1, 20, 64, 333])
def test_replayed_layers_are_the_calls(cuda, T):
    from mlp_step import Mlp
    eager, graph = (Mlp(512, 1408, rows=T, adapters=3, rank=8) for _ in range(2))
    g = cuda.Generator(device="cuda").manual_seed(T)
    adapter = cuda.randint(-1, 3, (T,), generator=g, device="cuda").int()
    graph.capture(T, adapter)
    for step in range(6):
        x, res = (cuda.randn(T, 512, generator=g, device="cuda").bfloat16() for _ in range(2))
        a, b = eager.step(x, res, adapter), graph.step(x, res, adapter)
        assert cuda.equal(a.view(cuda.int16), b.view(cuda.int16)) and cuda.equal(eager.residual, graph.residual), step
    assert eager.errors() == 0 and graph.errors() == 0


def test_rows_do_not_depend_on_the_batch(cuda):
    """A row's y is the same in a batch of any size (its sums are whole numbers)."""
    g = cuda.Generator(device="cuda").manual_seed(4)
    big = problem(cuda, g, 700, 5128, 5136)
    call(cuda, [big], 700)
    for T in (1, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 513):
        p = {**big, "T": T, "y": cuda.full((T + 2, 5128), 7.0, dtype=cuda.bfloat16, device="cuda")}
        call(cuda, [p], T)
        assert cuda.equal(p["y"][:T].view(cuda.int16), big["y"][:T].view(cuda.int16)), T


def test_calls_on_two_streams(cuda):
    """Two calls at once, each with its workspace."""
    g = cuda.Generator(device="cuda").manual_seed(5)
    for T in (1, 48, 300):
        ps = [problem(cuda, g, T, 5128, 5136) for _ in range(2)]
        for p in ps:
            call(cuda, [p], T)
        want = [p["y"].clone() for p in ps]
        streams, kept = [cuda.cuda.Stream() for _ in ps], []
        for p, s in zip(ps, streams):
            pr = problems([p])
            kept.append((pr, *workspace(cuda, pr, T)))
            p["y"].fill_(7.0)
        cuda.cuda.synchronize()
        for _ in range(10):
            for (pr, ws, size), s in zip(kept, streams):
                lora.w8_matmul(pr, T, ws, size, s.cuda_stream)
        cuda.cuda.synchronize()
        for p, y in zip(ps, want):
            assert cuda.equal(p["y"].view(cuda.int16), y.view(cuda.int16))


def test_one_workspace_for_both_kinds_of_products(cuda):
    from .test_gpu_w4 import check as check4
    from .test_gpu_w4 import problem as problem4
    g = cuda.Generator(device="cuda").manual_seed(6)
    for T in (5, 40, 200):
        p8, p4 = problem(cuda, g, T, 2056, 4096), problem4(cuda, g, T, 2048, 4096, 128, True)
        pr8 = problems([p8])
        pr4 = lora.w4_problems([(p4["x"], p4["y"], 4096, 2048, p4["codes"], p4["scales"], p4["zeros"], 2048, 4096, 128)])
        size = max(lora.w8_workspace_size(pr8, T), lora.w4_workspace_size(pr4, T))
        ws = cuda.empty(size, dtype=cuda.uint8, device="cuda")
        stream = cuda.cuda.current_stream().cuda_stream
        lora.kv_workspace_init(ws, size, stream)
        for _ in range(3):
            p8["y"][:T].fill_(0)
            p4["y"].fill_(0)
            lora.w8_matmul(pr8, T, ws, size, stream)
            lora.w4_matvec(pr4, T, ws, size, stream)
            check(cuda, p8)
            check4(cuda, p4)
        assert lora.get_device_error(ws, stream) == 0


def test_the_same_rows_for_several_projections(cuda):
    """Problems that share x share its copy, also when another one stands between them."""
    g = cuda.Generator(device="cuda").manual_seed(7)
    for T in (3, 70, 300):
        a, b = problem(cuda, g, T, 264, 528), problem(cuda, g, T, 264, 528)
        c, d = problem(cuda, g, T, 1032, 528, x=a), problem(cuda, g, T, 8, 528, x=b)
        call(cuda, [a, b, c, d], T)
        for p in (a, b, c, d):
            check(cuda, p)


@pytest.mark.parametrize("T,N,K,step", [(40, 14336, 4096, 20), (64, 14336, 4096, 100), (128, 4096, 14336, 1000), (300, 5128, 1040, 7)])
def test_the_workspace_serves_on_after_a_wait_that_ran_out(cuda, T, N, K, step):
    """A step of W that never comes: the timeout bit, and later calls on the same workspace are as on a fresh one."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    p = problem(cuda, g, T, N, K)
    pr = problems([p])
    ws, size = workspace(cuda, pr, T)
    stream = cuda.cuda.current_stream().cuda_stream
    lora.debug_w8_lost_step(pr, T, step, 5_000_000, ws, size, stream)
    assert lora.get_device_error(ws, stream) == 0x20
    assert bool((p["y"][T:] == 7).all())
    for _ in range(3):
        p["x"].copy_(cuda.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=cuda.int32))
        lora.w8_matmul(pr, T, ws, size, stream)
        assert lora.get_device_error(ws, stream) == 0
        check(cuda, p)



@pytest.mark.parametrize("step", [0, 200, 1000])
def test_the_workspace_serves_on_after_a_wait_in_one_of_many_tiles(cuda, step):
    """Several whole tiles a pair, the step that never comes in its first, a later or its last one."""
    g = cuda.Generator(device="cuda").manual_seed(step)
    T, ps = 300, []
    for N in (32776, 264, 8):
        ps.append(problem(cuda, g, T, N, 400, x=ps[0] if ps else None))
    pr = problems(ps)
    ws, size = workspace(cuda, pr, T)
    stream = cuda.cuda.current_stream().cuda_stream
    lora.debug_w8_lost_step(pr, T, step, 5_000_000, ws, size, stream)
    assert lora.get_device_error(ws, stream) == 0x20
    for _ in range(2):
        lora.w8_matmul(pr, T, ws, size, stream)
        assert lora.get_device_error(ws, stream) == 0
        for p in ps:
            check(cuda, p)


@pytest.mark.parametrize("T", [33, 64, 100, 130, 257, 300, 520, 700, 1030])
@pytest.mark.parametrize("K", [16, 400, 1040])
def test_many_tiles_of_projections_of_one_length(cuda, T, K):
    """Projections of one tile and of many, all with as many blocks of K: whole tiles, one pair's in several projections."""
    g = cuda.Generator(device="cuda").manual_seed(T + K)
    a = problem(cuda, g, T, 264, K)
    ps = [a, problem(cuda, g, T, 20488, K, x=a), problem(cuda, g, T, 8, K), problem(cuda, g, T, 16, K, x=a), problem(cuda, g, T, 5128, K, pad=8)]
    call(cuda, ps, T)
    for p in ps:
        check(cuda, p)


def test_lost_step_refusals(cuda):
    from heterogeneous_adapters_gb300 import _binding as B
    g = cuda.Generator(device="cuda").manual_seed(1)
    p = problem(cuda, g, 40, 8192, 4096)
    pr = problems([p])
    ws, size = workspace(cuda, pr, 40)
    for T, step, limit, want in ((8, 0, 5_000_000, B.LORA_EINVAL), (40, -1, 5_000_000, B.LORA_EINVAL), (40, 0, 1000, B.LORA_EINVAL),
                                 (40, 0, 3_000_000_000, B.LORA_ETOOBIG)):
        with pytest.raises(lora.LoraError) as e:
            lora.debug_w8_lost_step(pr, T, step, limit, ws, size, 0)
        assert e.value.status == want
    assert bool((p["y"] == 7).all())


@pytest.mark.parametrize("T", [1, 13, 40, 300])
def test_calls_that_feed_each_other_wait_for_each_other(cuda, T):
    """A chain of calls, each of which reads what the one before wrote and writes what the one before read, with
    and without a wait of the host between them, in a graph, and with W written by the kernel before."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    d, f = 1024, 2064
    h0 = cuda.randn(T, d, generator=g, device="cuda").bfloat16()
    weight = cuda.ones(d, dtype=cuda.bfloat16, device="cuda")
    up_w, down_w = codes(cuda, g, f, d), codes(cuda, g, d, f)
    up_s, down_s = (cuda.full((n,), 2.0 ** -12, device="cuda") for n in (f, d))
    h, y = cuda.empty_like(h0), cuda.zeros(T, d, dtype=cuda.bfloat16, device="cuda")
    xc, xs = cuda.empty(T, d, dtype=cuda.int8, device="cuda"), cuda.empty(T, device="cuda")
    a, ac, as_ = cuda.empty(T, f, dtype=cuda.bfloat16, device="cuda"), cuda.empty(T, f, dtype=cuda.int8, device="cuda"), cuda.empty(T, device="cuda")
    up_now = cuda.empty_like(up_w)
    norm = lora.Q8Norm(h, d, y, d, h, d, weight, 1e-5, d, lora.Q8Rows(xc, d, xs, None, 0, lora.LORA_Q8_X_HELD))
    gate = lora.Q8Gate(a, f, None, 0, lora.LORA_ACT_GELU, f, lora.Q8Rows(ac, f, as_, None, 0, lora.LORA_Q8_X_HELD))
    up = lora.w8_problems([(xc, xs, a, d, f, up_now, up_s, f, d)])
    down = lora.w8_problems([(ac, as_, y, f, d, down_w, down_s, d, f)])
    size = max(lora.w8_workspace_size(up, T), lora.w8_workspace_size(down, T))
    ws = cuda.empty(size, dtype=cuda.uint8, device="cuda")

    def steps(stream, between=lambda: None, n=20):
        h.copy_(h0)
        y.zero_()
        for i in range(n):
            up_now.copy_(up_w if i % 2 else up_w.flip(0))
            between()
            lora.q8_norm(norm, T, stream)
            between()
            lora.w8_matmul(up, T, ws, size, stream)
            between()
            lora.q8_gate(gate, T, stream)
            between()
            lora.w8_matmul(down, T, ws, size, stream)
            between()
            up_now.zero_()
            # W by the kernel right before
            up_now.copy_(up_w)
            lora.w8_matmul(up, T, ws, size, stream)
            between()

    side = cuda.cuda.Stream()
    with cuda.cuda.stream(side):
        s = side.cuda_stream
        lora.kv_workspace_init(ws, size, s)
        steps(s, side.synchronize)
        want = [t.clone() for t in (h, y, a, ac)]
        assert all(bool(cuda.isfinite(t.float()).all()) for t in want)
        for _ in range(5):
            steps(s)
            for t, w in zip((h, y, a, ac), want):
                assert cuda.equal(t, w)
        graph = cuda.cuda.CUDAGraph()
        side.synchronize()
        with cuda.cuda.graph(graph, stream=side):
            steps(side.cuda_stream)
        for _ in range(5):
            graph.replay()
            for t, w in zip((h, y, a, ac), want):
                assert cuda.equal(t, w)
        assert lora.get_device_error(ws, s) == 0


@pytest.mark.parametrize("T", [1, 13, 40, 300])
@pytest.mark.parametrize("first", ["call", "copy", "nothing"])
def test_branches_of_streams_that_join(cuda, T, first):
    """Calls behind two streams' work, eager and in one graph: each waits for both."""
    g = cuda.Generator(device="cuda").manual_seed(T)
    d, f = 1024, 2064
    x, gin = (cuda.randn(T, n, generator=g, device="cuda").bfloat16() for n in (d, f))
    weight = cuda.ones(d, dtype=cuda.bfloat16, device="cuda")
    up_w, down_w = codes(cuda, g, f, d), codes(cuda, g, d, f)
    up_s, down_s = (cuda.full((n,), 2.0 ** -12, device="cuda") for n in (f, d))
    xc, xs = cuda.empty(T, d, dtype=cuda.int8, device="cuda"), cuda.empty(T, device="cuda")
    ac, as_ = cuda.empty(T, f, dtype=cuda.int8, device="cuda"), cuda.empty(T, device="cuda")
    y1, y2 = cuda.empty(T, f, dtype=cuda.bfloat16, device="cuda"), cuda.empty(T, d, dtype=cuda.bfloat16, device="cuda")
    source = x.clone()
    norm = lora.Q8Norm(x, d, None, 0, None, 0, weight, 1e-5, d, lora.Q8Rows(xc, d, xs, None, 0, lora.LORA_Q8_X_HELD))
    gate = lora.Q8Gate(gin, f, None, 0, lora.LORA_ACT_SILU, f, lora.Q8Rows(ac, f, as_, None, 0, lora.LORA_Q8_X_HELD))
    both = lora.w8_problems([(xc, xs, y1, d, f, up_w, up_s, f, d), (ac, as_, y2, f, d, down_w, down_s, d, f)])
    size = lora.w8_workspace_size(both, T)
    ws = cuda.empty(size, dtype=cuda.uint8, device="cuda")
    main, side = cuda.cuda.Stream(), cuda.cuda.Stream()
    outs = (xc, xs, ac, as_, y1, y2)

    def run(wait=False):
        if first == "copy":
            x.copy_(source)
        elif first == "call":
            lora.q8_norm(norm, T, main.cuda_stream)
        side.wait_stream(main)
        lora.q8_gate(gate, T, side.cuda_stream)
        lora.q8_norm(norm, T, main.cuda_stream)
        main.wait_stream(side)
        if wait:
            main.synchronize()
        lora.w8_matmul(both, T, ws, size, main.cuda_stream)
        side.wait_stream(main)
        lora.q8_gate(gate, T, side.cuda_stream)
        main.wait_stream(side)
        lora.w8_matmul(both, T, ws, size, main.cuda_stream)

    with cuda.cuda.stream(main):
        lora.kv_workspace_init(ws, size, main.cuda_stream)
        run(True)
        main.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        run()
        assert all(cuda.equal(t, w) for t, w in zip(outs, want))
        graph = cuda.cuda.CUDAGraph()
        main.synchronize()
        with cuda.cuda.graph(graph, stream=main):
            run()
        for _ in range(3):
            for t in outs:
                t.zero_()
            graph.replay()
            assert all(cuda.equal(t, w) for t, w in zip(outs, want))
        assert lora.get_device_error(ws, main.cuda_stream) == 0
