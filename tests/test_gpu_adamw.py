"""AdamW on the GPU against the fp64 oracle.

8-bit codes and exponents are defined to the bit and compared for equality.  fp32 results are
compared within bounds that count the roundings (u = 2^-24, half a step):
  m, v  two coefficients, two products, one sum (v: one product more): 6 u of the terms' sizes
  p     p (1 - lr wd): 3 u; the step: m and v as above (v halves under the root), root, two
        products, a sum, a quotient, a product and two rounded coefficients: 20 u of its size;
        where eps dominates the denominator the same holds.  bf16 adds half a step of the result
        when rounded to nearest, a whole one when rounded stochastically.
"""

import copy
import math

import numpy as np
import pytest
import torch

from oracle import adamw

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def _np(t):
    return t.detach().double().cpu().numpy()


def _flat(t):
    """The elements in the order of memory."""
    return t.detach().as_strided((t.numel(),), (1,), t.storage_offset())


class Reference:
    """One parameter in the oracle: states are read from the optimizer's own after each step."""

    def __init__(self, p, ident, bits, rounding, seed):
        self.ident, self.bits, self.rounding, self.seed = ident, bits, rounding, seed
        n = p.numel()
        self.t = 0
        self.m = np.zeros(n) if bits == 32 else (np.zeros(n, np.uint8), np.zeros(-(-n // 128), np.uint8))
        self.v = copy.deepcopy(self.m)

    def step(self, before, g, p, state, hyper, bf16):
        """Checks p and its state after a step from `before` with the gradient g (memory order)."""
        (b1, b2), lr, eps, wd = hyper["betas"], hyper["lr"], hyper["eps"], hyper["weight_decay"]
        self.t += 1
        n = len(g)
        if self.bits == 8:
            m0, v0 = adamw.decode(*self.m, True), adamw.decode(*self.v, False)
        else:
            m0, v0 = self.m, self.v
        m, v = adamw.moments(m0, v0, g, b1, b2)
        want = adamw.parameter(before, m, v, self.t, lr, b1, b2, eps, wd)
        size = lr / (1 - b1 ** self.t) * (np.abs(b1 * m0) + np.abs((1 - b1) * g)) / (np.sqrt(v) / math.sqrt(1 - b2 ** self.t) + eps)
        size = np.where(np.isfinite(size), size, 0.0)
        bound = 3 * U * np.abs(before) + 20 * U * size + 2.0 ** -148
        got = _np(_flat(p))
        if bf16:
            step = 2.0 ** -8 if self.rounding == "rn" else 2.0 ** -7
            bound = bound + step * (np.abs(want) + bound)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        fine = ~np.isnan(want)
        assert np.all(np.abs(got - want)[fine] <= bound[fine])
        em, ev = _flat(state["exp_avg"]).cpu().numpy(), _flat(state["exp_avg_sq"]).cpu().numpy()
        if self.bits == 32:
            bm = 6 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g)) + 2.0 ** -148
            bv = 6 * U * (b2 * v0 + (1 - b2) * g * g) + 2.0 ** -148
            ok = np.isfinite(m)
            assert np.all(np.abs(em - m)[ok] <= bm[ok]) and np.all(np.abs(ev - v)[ok] <= bv[ok])
            self.m, self.v = em.astype(np.float64), ev.astype(np.float64)
            return
        w = adamw.words(self.seed, self.ident, 0, self.t, n) if self.rounding == "sr" else None
        bad = ~(np.isfinite(m) & np.isfinite(v))
        m, v = np.where(bad, np.nan, m), np.where(bad, np.nan, v)
        self.m = adamw.encode(m, True, None if w is None else w & np.uint64(0xFFFF))
        self.v = adamw.encode(v, False, None if w is None else w >> np.uint64(16))
        assert np.array_equal(em, self.m[0]) and np.array_equal(ev, self.v[0])
        assert np.array_equal(state["exp_avg_exponent"].cpu().numpy(), self.m[1])
        assert np.array_equal(state["exp_avg_sq_exponent"].cpu().numpy(), self.v[1])


SIZES = [(1,), (3,), (127,), (128,), (129,), (2047,), (2049,), (5, 77), (64, 130), (300, 301)]


def _params(sizes, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.nn.Parameter((0.1 * torch.randn(*s, generator=g)).to(dtype).cuda()) for s in sizes]


def _gradient(p, seed, scale=1e-2):
    g = torch.Generator().manual_seed(seed)
    x = scale * torch.randn(p.numel(), generator=g) * torch.exp(2 * torch.randn(p.numel(), generator=g))
    x[::7] = 0
    return x.reshape(p.shape).to(p.dtype).to(p.device)


def _run(opt, params, refs, steps, hyper, grads=_gradient, first=0):
    for s in range(first, first + steps):
        before = [_np(_flat(p)) for p in params]
        for i, p in enumerate(params):
            p.grad = grads(p, 1000 * s + i)
        opt.step()
        for i, p in enumerate(params):
            g = torch.empty_like(p, memory_format=torch.preserve_format).copy_(p.grad)
            refs[i].step(before[i], _np(_flat(g)), p, opt.state[p], hyper, p.dtype == torch.bfloat16)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("rounding", ["rn", "sr"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_match_the_oracle(metis_lib, bits, rounding, dtype):
    from spectral_quantized_gemm_b200.optim import AdamW
    params = _params(SIZES, dtype, 1)
    opt = AdamW(params, state_bits=bits, rounding=rounding, seed=(3 << 40) + 5, **HYPER)
    refs = [Reference(p, i, bits, rounding, (3 << 40) + 5) for i, p in enumerate(params)]
    _run(opt, params, refs, 5, HYPER)


@pytest.mark.parametrize("bits", [32, 8])
def test_hundreds_of_tensors_groups_and_missing_gradients(metis_lib, bits):
    """More tensors than one launch takes; two groups with their own options; gradients that come and go."""
    from spectral_quantized_gemm_b200.optim import AdamW
    params = _params([(1 + 37 * i % 900,) for i in range(900)], torch.float32, 2)
    other = dict(lr=1e-4, betas=(0.5, 0.9), eps=1e-3, weight_decay=0.0)
    opt = AdamW([{"params": params[:850]}, {"params": params[850:], "state_bits": 40 - bits, **other}], state_bits=bits,
                rounding="sr", seed=9, **HYPER)
    refs = [Reference(p, i, bits if i < 850 else 40 - bits, "sr", 9) for i, p in enumerate(params)]
    for s in range(3):
        live = [i for i in range(900) if (i + s) % 3]
        before = {i: _np(params[i]) for i in range(900)}
        for i, p in enumerate(params):
            p.grad = _gradient(p, s * 1000 + i) if i in set(live) else None
        opt.step()
        for i in range(900):
            if i in set(live):
                refs[i].step(before[i], _np(params[i].grad), params[i], opt.state[params[i]], HYPER if i < 850 else other, False)
            else:
                assert np.array_equal(_np(params[i]), before[i])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_views_strides_and_neighbours(metis_lib, bits, dtype):
    """Parameters that start anywhere in a buffer, transposed ones, gradients with other strides."""
    from spectral_quantized_gemm_b200.optim import AdamW
    buf = (0.1 * torch.randn(5000, generator=torch.Generator().manual_seed(3))).to(dtype).cuda()
    keep = buf.clone()
    params = [torch.nn.Parameter(buf[1:1 + 333]), torch.nn.Parameter(buf[1001:1001 + 40 * 50].view(40, 50).t()),
              torch.nn.Parameter(buf[4003:4003 + 130].view(1, 130, 1))]
    opt = AdamW(params, state_bits=bits, rounding="sr", **HYPER)
    refs = [Reference(p, i, bits, "sr", 0) for i, p in enumerate(params)]

    def grads(p, seed):
        g = _gradient(p, seed)
        return g.contiguous() if seed % 2 else torch.cat([g, g], -1)[..., :g.shape[-1]]

    _run(opt, params, refs, 3, HYPER, grads)
    gaps = torch.ones(5000, dtype=torch.bool, device="cuda")
    for p in params:
        gaps[p.storage_offset():p.storage_offset() + p.numel()] = False
    assert torch.equal(buf[gaps], keep[gaps])


def test_broadcast_gradient(metis_lib):
    from spectral_quantized_gemm_b200.optim import AdamW
    params = _params([(30, 40)], torch.float32, 4)
    opt = AdamW(params, state_bits=8, rounding="rn", **HYPER)
    refs = [Reference(params[0], 0, 8, "rn", 0)]
    _run(opt, params, refs, 2, HYPER, lambda p, s: torch.full((1, 1), 0.25, device="cuda").expand(30, 40))


@pytest.mark.parametrize("bits", [32, 8])
def test_extreme_gradients(metis_lib, bits):
    """Zeros, subnormals, the largest values, NaN and infinities, and the status they raise."""
    from spectral_quantized_gemm_b200.linear import _shared_context
    from spectral_quantized_gemm_b200.optim import AdamW
    lib, _ = _shared_context(torch.device("cuda", 0))
    lib.poll_device_status()
    params = _params([(700,)], torch.float32, 5)
    opt = AdamW(params, state_bits=bits, rounding="rn", **HYPER)
    refs = [Reference(params[0], 0, bits, "rn", 0)]
    fine = torch.cat([torch.tensor([0.0, -0.0, 1e-45, -1e-40, 1e-20, 1e18, -1e18, 1.0]), torch.zeros(400), torch.full((292,), 1e-12)])
    _run(opt, params, refs, 3, HYPER, lambda p, s: fine.cuda() * (1 if s < 2000 else -1))
    assert lib.poll_device_status() == 0
    worse = fine.clone()
    worse[10], worse[200], worse[201] = float("nan"), float("inf"), -float("inf")
    _run(opt, params, refs, 1, HYPER, lambda p, s: worse.cuda(), first=3)
    assert lib.poll_device_status() == metis_lib.DEV_NONFINITE
    assert torch.isnan(params[0]).sum() == 3
    if bits == 8:                                     # the others go on as if nothing had happened
        params[0].data[torch.isnan(params[0])] = 0
        _run(opt, params, refs, 1, HYPER, lambda p, s: fine.cuda(), first=4)


def test_square_of_a_huge_gradient_saturates(metis_lib):
    from spectral_quantized_gemm_b200.optim import AdamW
    p = torch.nn.Parameter(torch.ones(128, device="cuda"))
    opt = AdamW([p], state_bits=8, rounding="rn", lr=1e-2, weight_decay=0.0)
    p.grad = torch.full_like(p, 1e-3)
    p.grad[5] = 3e38
    opt.step()
    assert torch.isfinite(p).all() and opt.state[p]["exp_avg_sq"][5] == 255
    assert opt.state[p]["exp_avg_sq_exponent"].item() == 254


def test_a_second_moment_follows_only_with_stochastic_rounding(metis_lib):
    """With beta2 = 0.999 one step moves v by a thousandth, far below half a code step (1/16): to
    nearest it stays, stochastically it follows on average.  v decays from 1 to 0.999^400 = 0.67 in
    128 * 64 elements; each element's error is below two code steps (1/8 of its value each way), so
    the mean's standard deviation is below 0.25 / sqrt(8192) < 0.003: 0.02 is seven of those.  One
    element a block is held at 1 by its gradient, so that the block's exponent does not move."""
    from spectral_quantized_gemm_b200.optim import AdamW
    mean = {}
    for rounding in ("rn", "sr"):
        p = torch.nn.Parameter(torch.zeros(128 * 64, device="cuda"))
        opt = AdamW([p], state_bits=8, rounding=rounding, betas=(0.0, 0.999), lr=0.0)
        held = torch.zeros_like(p)
        held[::128] = 1.0
        p.grad = held
        opt.step()
        state = opt.state[p]
        state["exp_avg_sq"].fill_(31 * 8)             # (8 + 0) 2^30 u = 2^(E - 127) = 1
        state["exp_avg_sq_exponent"].fill_(127)
        for _ in range(400):
            opt.step()
        codes, E = state["exp_avg_sq"].cpu().numpy(), state["exp_avg_sq_exponent"].cpu().numpy()
        v = adamw.decode(codes, E, False).reshape(-1, 128)[:, 1:]
        mean[rounding] = v.mean()
    assert mean["rn"] == 1.0
    assert abs(mean["sr"] - 0.999 ** 400) < 0.02


def test_repeated_runs_give_the_same_bits(metis_lib):
    from spectral_quantized_gemm_b200.optim import AdamW
    results = []
    for seed in (1, 1, 2):
        params = _params([(1000,), (77, 9)], torch.bfloat16, 6)
        opt = AdamW(params, state_bits=8, rounding="sr", seed=seed, **HYPER)
        for s in range(3):
            for i, p in enumerate(params):
                p.grad = _gradient(p, 10 * s + i)
            opt.step()
        results.append([p.detach().clone() for p in params] + [opt.state[p]["exp_avg"].clone() for p in params])
    assert all(torch.equal(a, b) for a, b in zip(results[0], results[1]))
    assert not all(torch.equal(a, b) for a, b in zip(results[0], results[2]))


@pytest.mark.parametrize("capturable", [False, True])
def test_checkpoint_resumes_bit_for_bit(metis_lib, capturable):
    import io
    from spectral_quantized_gemm_b200.optim import AdamW

    def make():
        params = _params([(1000,), (40, 30)], torch.float32, 7)
        return params, AdamW([{"params": params[:1]}, {"params": params[1:], "state_bits": 32}], state_bits=8, seed=4,
                             capturable=capturable, **HYPER)

    def train(params, opt, first, steps):
        for s in range(first, first + steps):
            for i, p in enumerate(params):
                p.grad = _gradient(p, 10 * s + i)
            opt.step()

    params, opt = make()
    train(params, opt, 0, 3)
    buf = io.BytesIO()
    torch.save({"opt": opt.state_dict(), "p": [p.detach().cpu() for p in params]}, buf)
    train(params, opt, 3, 3)
    for where in ("cuda", "cpu"):
        buf.seek(0)
        saved = torch.load(buf, map_location=where)
        again, opt2 = make()
        for p, q in zip(again, saved["p"]):
            p.data.copy_(q)
        opt2.load_state_dict(saved["opt"])
        assert opt2.state[again[0]]["exp_avg"].dtype == torch.uint8
        train(again, opt2, 3, 3)
        for p, q in zip(params, again):
            assert torch.equal(p, q)
            for k, v in opt.state[p].items():
                w = opt2.state[q][k]
                assert torch.equal(v, w) if isinstance(v, torch.Tensor) else v == w


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_count_and_schedule_on_the_device(metis_lib, bits):
    from spectral_quantized_gemm_b200.optim import AdamW
    lr = torch.tensor(1e-2, device="cuda")
    params, plain = _params(SIZES, torch.float32, 8), _params(SIZES, torch.float32, 8)
    hyper = {k: v for k, v in HYPER.items() if k != "lr"}
    opt = AdamW(params, lr=lr, state_bits=bits, seed=6, capturable=True, **hyper)
    want = AdamW(plain, lr=1e-2, state_bits=bits, seed=6, **hyper)
    for i, (p, q) in enumerate(zip(params, plain)):
        p.grad, q.grad = _gradient(p, i), _gradient(q, i)
    fresh = AdamW([torch.nn.Parameter(torch.zeros(4, device="cuda"))], capturable=True)
    fresh.param_groups[0]["params"][0].grad = torch.ones(4, device="cuda")
    opt.step()
    want.step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError):
            fresh.step()                              # no states yet
        with pytest.raises(RuntimeError):
            want.step()                               # not capturable
        opt.step()
    for s in range(4):
        rate = 1e-2 / (s + 1)
        lr.fill_(rate)
        want.param_groups[0]["lr"] = float(np.float32(rate))
        for i, (p, q) in enumerate(zip(params, plain)):
            p.grad.copy_(_gradient(p, 100 * s + i))
            q.grad.copy_(p.grad)
        graph.replay()
        want.step()
    torch.cuda.synchronize()
    assert opt.param_groups[0]["step_count"].item() == 5
    for p, q in zip(params, plain):
        assert torch.equal(p, q)
        assert torch.equal(opt.state[p]["exp_avg_sq"], want.state[q]["exp_avg_sq"])


def test_what_moves_between_steps_is_followed(metis_lib):
    """Steps after the first use what the last one gathered, unless something lies elsewhere now: new
    gradients, a parameter or state with new memory, replaced states, a gradient in another order, a
    missing one, changed options."""
    import copy
    from spectral_quantized_gemm_b200.optim import AdamW
    params = _params([(500,), (30, 40), (130,)], torch.float32, 11)
    hyper = dict(HYPER)
    opt = AdamW(params, state_bits=8, rounding="rn", **hyper)
    refs = [Reference(p, i, 8, "rn", 0) for i, p in enumerate(params)]

    def step(seed, hyper=hyper):
        _run(opt, params, refs, 1, hyper, first=seed)

    for s in range(3):
        step(s)
    with torch.no_grad():
        params[0].data = params[0].data.clone()
    step(3)
    opt.state[params[1]]["exp_avg"] = opt.state[params[1]]["exp_avg"].clone()
    step(4)
    opt.state[params[2]]["exp_avg_exponent"].data = opt.state[params[2]]["exp_avg_exponent"].clone()
    step(5)
    opt.state[params[0]] = copy.deepcopy(opt.state[params[0]])
    step(6)
    opt.load_state_dict(opt.state_dict())
    step(7)
    hyper = dict(hyper, lr=1e-2, betas=(0.8, 0.9), weight_decay=0.0)
    opt.param_groups[0].update(hyper)
    step(8, hyper)
    # a gradient in another order, then the usual one
    _run(opt, params, refs, 1, hyper, lambda p, s: _gradient(p, s).t().contiguous().t() if p.dim() == 2 else _gradient(p, s), first=9)
    step(10, hyper)
    # a parameter without a gradient falls a step behind and keeps its own count
    before = [_np(_flat(p)) for p in params]
    for i, p in enumerate(params):
        p.grad = None if i == 1 else _gradient(p, 900 + i)
    opt.step()
    for i in (0, 2):
        refs[i].step(before[i], _np(params[i].grad), params[i], opt.state[params[i]], hyper, False)
    assert np.array_equal(_np(_flat(params[1])), before[1])
    step(12, hyper)
    step(13, hyper)
    assert [opt.state[p]["step"] for p in params] == [14, 13, 14]


def test_copies_of_the_optimizer_keep_their_stream(metis_lib):
    import copy
    import pickle
    from spectral_quantized_gemm_b200.optim import AdamW
    results = []
    for how in (lambda x: x, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))):
        params = _params([(300,)], torch.float32, 12)
        opt = AdamW(params, state_bits=8, seed=99, **HYPER)
        for s in range(4):
            if s == 2:
                opt = how(opt)
                params = opt.param_groups[0]["params"]
            params[0].grad = _gradient(params[0], s)
            opt.step()
        results.append((params[0].detach().clone(), opt.state[params[0]]["exp_avg_sq"].clone()))
    for p, v in results[1:]:
        assert torch.equal(p, results[0][0]) and torch.equal(v, results[0][1])


def test_a_step_is_seen_by_autograd(metis_lib):
    """A parameter saved for a backward pass and then stepped: the pass is refused, as with torch's own."""
    from spectral_quantized_gemm_b200.optim import AdamW
    p = torch.nn.Parameter(torch.ones(8, device="cuda"))
    opt = AdamW([p])
    for _ in range(3):
        loss = (p * p).sum()
        p.grad = torch.ones_like(p)
        opt.step()
        with pytest.raises(RuntimeError):
            loss.backward()


def test_more_than_two_to_the_31_elements(metis_lib):
    from spectral_quantized_gemm_b200.optim import AdamW
    n = 2 ** 31 + 300
    p = torch.nn.Parameter(torch.zeros(n, dtype=torch.bfloat16, device="cuda"))
    p.grad = torch.zeros_like(p)
    tail = 555
    p.grad[-tail:] = _gradient(p[-tail:], 1)
    opt = AdamW([p], state_bits=8, rounding="sr", seed=2, **HYPER)
    before = _np(p[-tail:])
    opt.step()
    m, v = adamw.moments(np.zeros(tail), np.zeros(tail), _np(p.grad[-tail:]), *HYPER["betas"])
    want = adamw.parameter(before, m, v, 1, HYPER["lr"], *HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
    assert np.all(np.abs(_np(p[-tail:]) - want) <= 2.0 ** -7 * np.abs(want) * (1 + 1e-3) + 1e-9)
    first = n - n % 128 - 256                              # whole blocks from here
    words = adamw.philox.stream_words(2, adamw.philox.tag(0, 4, 0), 1, np.arange(first // 4, -(-n // 4), dtype=np.uint64))
    words = words.reshape(-1)[:n - first]
    g = _np(p.grad[first:])
    m, v = adamw.moments(np.zeros(len(g)), np.zeros(len(g)), g, *HYPER["betas"])
    assert np.array_equal(opt.state[p]["exp_avg"][first:].cpu().numpy(), adamw.encode(m, True, words & np.uint64(0xFFFF))[0])
    assert np.array_equal(opt.state[p]["exp_avg_sq"][first:].cpu().numpy(), adamw.encode(v, False, words >> np.uint64(16))[0])
    assert (opt.state[p]["exp_avg"][:first:1 << 20] == 0).all()


@pytest.mark.parametrize("bits,rounding", [(8, "sr"), (8, "rn"), (32, "sr")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_tensors_aligned_or_not_take_the_same_step(metis_lib, bits, rounding, dtype):
    """Several state blocks a warp (whole chunks, and the ragged last one): arrays that start on 16 bytes
    and arrays that start between take different loads to the same bits."""
    from spectral_quantized_gemm_b200.optim import AdamW
    n = 6_000_077
    g = torch.Generator(device="cuda").manual_seed(5)
    start = torch.randn(n, device="cuda", generator=g).to(dtype)
    params = [torch.nn.Parameter(start.clone()), torch.nn.Parameter(torch.empty(n + 1, dtype=dtype, device="cuda")[1:].copy_(start))]
    opts = [AdamW([p], state_bits=bits, rounding=rounding, **HYPER) for p in params]
    for _ in range(3):
        grad = (1e-2 * torch.randn(n, device="cuda", generator=g)).to(dtype)
        for p, opt in zip(params, opts):
            p.grad = grad if p is params[0] else torch.empty(n + 1, dtype=dtype, device="cuda")[1:].copy_(grad)
            opt.step()
    assert torch.equal(*[p.detach() for p in params])
    for key in opts[0].state[params[0]]:
        if key != "step":
            assert torch.equal(*[opt.state[p][key] for p, opt in zip(params, opts)]), key


def test_refusals(metis_lib):
    from spectral_quantized_gemm_b200.optim import AdamW
    p = torch.nn.Parameter(torch.zeros(300, device="cuda"))
    opt = AdamW([p], state_bits=8, **HYPER)
    p.grad = torch.ones(300, device="cuda").to_sparse()
    with pytest.raises(ValueError):
        opt.step()
    p.grad = torch.ones(300, device="cuda")
    opt.step()
    good = dict(opt.state[p])
    for name, bad in (("exp_avg", good["exp_avg"].float()), ("exp_avg", good["exp_avg"][:200]),
                      ("exp_avg_sq_exponent", good["exp_avg_sq_exponent"][:2]), ("exp_avg_exponent", good["exp_avg_exponent"].int()),
                      ("exp_avg_sq", good["exp_avg_sq"].cpu()), ("exp_avg_exponent", good["exp_avg_exponent"].cpu())):
        opt.state[p] = {**good, name: bad}
        with pytest.raises(ValueError):
            opt.step()
    opt.state[p] = good
    twin = torch.nn.Parameter(p.detach())                  # another parameter on the same memory
    twin.grad = p.grad.clone()
    with pytest.raises(ValueError):
        AdamW([p, twin], **HYPER).step()
    opt.param_groups[0]["state_bits"] = 32
    with pytest.raises(ValueError):
        opt.step()

    ctx = metis_lib.Context()
    entry = metis_lib.AdamWTensor(p.data_ptr(), p.grad.data_ptr(), good["exp_avg"].data_ptr(), good["exp_avg_sq"].data_ptr(),
                                  good["exp_avg_exponent"].data_ptr(), good["exp_avg_sq_exponent"].data_ptr(), 300, 0, 0)
    fine = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, state_bits=8)

    def status(n=1, **kw):
        e = metis_lib.AdamWTensor.from_buffer_copy(entry)
        for k in list(kw):
            if hasattr(e, k):
                setattr(e, k, kw.pop(k))
        with pytest.raises(metis_lib.MetisError) as err:
            ctx.adamw_step(metis_lib.ctypes.byref(e), n, **{**fine, **kw})
        return err.value.status

    before = p.detach().clone()
    for kw in (dict(state_bits=16), dict(rounding=2), dict(beta1=1.0), dict(beta2=-0.1), dict(beta2=float("nan")), dict(eps=-1.0),
               dict(lr=float("inf")), dict(weight_decay=float("nan")), dict(step=0), dict(p=None), dict(g=None), dict(m=None),
               dict(v_exponent=None), dict(dtype=3), dict(id=1 << 24), dict(n=-1)):
        assert status(**kw) in (1, 2), kw
    assert status(p=p.data_ptr() + 2) == 3 and status(g=p.grad.data_ptr() + 1) == 3
    assert status(state_bits=32, m=good["exp_avg"].data_ptr() + 1) == 3
    with pytest.raises(ValueError):
        ctx.adamw_step(metis_lib.ctypes.byref(entry), 1, lr_dev=torch.zeros(1), **fine)
    assert torch.equal(p, before)
    ctx.adamw_step(None, 0, **fine)                        # nothing to do
    entry.n = 0
    ctx.adamw_step(metis_lib.ctypes.byref(entry), 1, **fine)
    assert torch.equal(p, before)
    ctx.close()


def test_layers_and_optimizer_together(metis_lib):
    """A training run of two layers, one on 8-bit integers and one on NVFP4, whose fp32 master weights
    AdamW steps with 8-bit states; after each step the integer layer's gradient and the step are
    checked against the oracle, and at the end the frozen layer serves what the trained one computes."""
    from oracle import int8
    from spectral_quantized_gemm_b200.int8_linear import Int8Linear
    from spectral_quantized_gemm_b200.linear import MetisLinear
    from spectral_quantized_gemm_b200.optim import AdamW
    torch.manual_seed(0)
    up, down = Int8Linear(256, 512, device="cuda"), MetisLinear(512, 256, device="cuda")
    opt = AdamW([{"params": up.parameters()}, {"params": down.parameters(), "state_bits": 32}], state_bits=8, seed=1, **HYPER)
    ref = Reference(up.weight, 0, 8, "sr", 1)
    for s in range(4):
        x = torch.randn(256, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(s)).bfloat16()
        seen = []
        h = up(x)
        h.register_hook(lambda d: seen.append(d.clone()))
        out = down(torch.nn.functional.gelu(h))
        loss = out.float().square().mean()
        opt.zero_grad()
        loss.backward()
        dw = int8.product(*int8.quantize_rows(_np(x).T), *int8.quantize_rows(_np(seen[0]).T))
        assert torch.equal(up.weight.grad.cpu(), torch.from_numpy(dw))
        before, g = _np(_flat(up.weight)), _np(_flat(up.weight.grad))
        was = down.weight.detach().clone()
        opt.step()
        ref.step(before, g, up.weight, opt.state[up.weight], HYPER, False)
        assert not torch.equal(was, down.weight) and torch.isfinite(down.weight).all()
    with torch.no_grad():
        want = up(x)
        assert torch.equal(up.freeze()(x), want)


def _cancelling(blocks, b1, seed):
    """First moments of a block's top octave and gradients that cancel them to 2^-7 .. 2^-26 in one step (deeper from
    block to block), a few whole cancellations among them."""
    rng = np.random.default_rng(seed)
    m = rng.integers(8, 16, (blocks, 128)) / 16.0 * rng.choice([-1.0, 1.0], (blocks, 128))
    depth = np.linspace(5, 24, blocks)[:, None] + rng.uniform(0, 16, (blocks, 128)) * (rng.random((blocks, 128)) < 0.7)
    g = -(b1 * m / (1 - b1)) * (1 + rng.choice([-1.0, 1.0], m.shape) * 2.0 ** -np.minimum(depth, 26))
    return m.reshape(-1), g.astype(np.float32).reshape(-1)


@pytest.mark.parametrize("rounding", ["rn", "sr"])
@pytest.mark.parametrize("b1", [0.85, 0.9, 0.99])
def test_first_moments_that_cancel(metis_lib, rounding, b1):
    from spectral_quantized_gemm_b200.optim import AdamW
    hyper = dict(HYPER, betas=(b1, 0.99))
    starts = [(np.array([0.34375]), np.array([-1.947916865], np.float32))] + [_cancelling(60, b1, s) for s in range(4)]
    m1, g1 = _cancelling(200, b1, 9)
    starts += [(m1[i:i + 1], g1[i:i + 1]) for i in range(0, 128 * 200, 128)]           # blocks of one element
    params = [torch.nn.Parameter(torch.ones(len(m), device="cuda")) for m, _ in starts]
    opt = AdamW(params, state_bits=8, rounding=rounding, seed=3, **hyper)
    refs = [Reference(p, i, 8, rounding, 3) for i, p in enumerate(params)]
    for p, ref, (m, g) in zip(params, refs, starts):
        ref.m, ref.v = adamw.encode(m, True), adamw.encode(m * m, False)
        assert np.array_equal(adamw.decode(*ref.m, True), m)
        opt.state[p] = {"step": 0, "exp_avg": torch.from_numpy(ref.m[0]).cuda(), "exp_avg_exponent": torch.from_numpy(ref.m[1]).cuda(),
                        "exp_avg_sq": torch.from_numpy(ref.v[0]).cuda(), "exp_avg_sq_exponent": torch.from_numpy(ref.v[1]).cuda()}
        p.grad = torch.from_numpy(g).cuda()
    before = [_np(p) for p in params]
    opt.step()
    for p, ref, b, (m, g) in zip(params, refs, before, starts):
        ref.step(b, g.astype(np.float64), p, opt.state[p], hyper, False)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_whose_square_leaves_fp32(metis_lib, bits, dtype):
    """g^2 is beyond fp32 from 1.8e19 on, (1 - b2) g^2 is not."""
    from spectral_quantized_gemm_b200.optim import AdamW
    hyper = dict(HYPER, betas=(0.9, 0.999))
    params = _params([(700,)], dtype, 5)
    opt = AdamW(params, state_bits=bits, rounding="rn", **hyper)
    refs = [Reference(params[0], 0, bits, "rn", 0)]
    g = torch.cat([torch.tensor([0.0, 2e19, -2e19, 1e20, -1e20, 1e18, 3e17, 1.0]), torch.zeros(300), torch.full((392,), 4e19)])
    _run(opt, params, refs, 3, hyper, lambda p, s: (g if s < 2000 else -0.5 * g).to(dtype).cuda())
    assert torch.isfinite(params[0]).all() and all(torch.isfinite(s.float()).all() for s in opt.state[params[0]].values() if isinstance(s, torch.Tensor))


@pytest.mark.parametrize("bits", [32, 8])
def test_counts_follow_a_change_of_capturable(metis_lib, bits):
    from spectral_quantized_gemm_b200.optim import AdamW
    runs = []
    for change in (False, True):
        params = _params([(500,), (30, 40)], torch.float32, 14)
        opt = AdamW(params, state_bits=bits, seed=8, **HYPER)
        for s in range(9):
            if change and s in (3, 6):
                opt.param_groups[0]["capturable"] = s == 3
            for i, p in enumerate(params):
                p.grad = _gradient(p, 10 * s + i)
            opt.step()
        runs.append((params, opt))
    (a, opt_a), (b, opt_b) = runs
    for p, q in zip(a, b):
        assert torch.equal(p, q) and opt_b.state[q]["step"] == opt_a.state[p]["step"] == 9
        assert torch.equal(opt_a.state[p]["exp_avg_sq"], opt_b.state[q]["exp_avg_sq"])
    b[0].grad, b[1].grad = _gradient(b[0], 1), None
    opt_b.step()
    opt_b.param_groups[0]["capturable"] = True             # ten steps and nine: no count for both
    b[1].grad = _gradient(b[1], 2)
    with pytest.raises(ValueError):
        opt_b.step()


@pytest.mark.parametrize("bits", [32, 8])
def test_replaced_states_restart_the_count_on_the_device(metis_lib, bits):
    from spectral_quantized_gemm_b200.optim import AdamW
    params, plain = _params([(500,)], torch.float32, 15), _params([(500,)], torch.float32, 15)
    opts = [AdamW(params, state_bits=bits, seed=8, capturable=True, **HYPER), AdamW(plain, state_bits=bits, seed=8, **HYPER)]
    for s in range(6):
        for p, opt in zip((params[0], plain[0]), opts):
            if s == 3:
                opt.state.clear()
            p.grad = _gradient(p, s)
            opt.step()
    assert torch.equal(params[0], plain[0]) and opts[0].param_groups[0]["step_count"].item() == 3


@pytest.mark.parametrize("capturable", [False, True])
def test_a_refused_step_is_not_counted(metis_lib, capturable):
    from spectral_quantized_gemm_b200.optim import AdamW
    p = torch.nn.Parameter(torch.ones(300, device="cuda"))
    opt = AdamW([p], capturable=capturable, **HYPER)

    def count():
        return opt.param_groups[0]["step_count"].item() if capturable else opt.state[p]["step"]

    for steps in (1, 2):                                   # a plan is there from the second on
        p.grad = torch.ones_like(p)
        opt.step()
        for fresh in (False, True):
            opt.param_groups[0]["eps"] = -1.0
            p.grad = torch.ones_like(p)
            if fresh:
                opt._plans.clear()
            before = p.detach().clone()
            with pytest.raises(metis_lib.MetisError):
                opt.step()
            opt.param_groups[0]["eps"] = 1e-8
            assert count() == steps and torch.equal(p, before)


@pytest.mark.parametrize("bits", [32, 8])
def test_smallest_eps(metis_lib, bits):
    """An eps below fp32's smallest number still keeps 0 / (0 + eps) at 0."""
    from spectral_quantized_gemm_b200.optim import AdamW
    for eps in (1e-50, 1e-45, 1e-40, 1e-300):
        p = torch.nn.Parameter(torch.ones(300, device="cuda"))
        opt = AdamW([p], lr=1e-2, eps=eps, weight_decay=0.0, state_bits=bits, rounding="rn")
        p.grad = torch.zeros_like(p)
        p.grad[::3] = 1e-3
        opt.step()
        opt.step()
        assert (p[1::3] == 1).all() and torch.isfinite(p).all() and (p[::3] < 1).all()


def test_checkpoint_of_a_learning_rate_on_the_device(metis_lib):
    import io
    from spectral_quantized_gemm_b200.optim import AdamW
    hyper = {k: v for k, v in HYPER.items() if k != "lr"}

    def make():
        params = _params([(300,)], torch.float32, 16)
        return params[0], AdamW(params, lr=torch.tensor(1e-2, device="cuda"), state_bits=8, capturable=True, **hyper)

    def train(p, opt, first):
        for s in range(first, first + 2):
            opt.param_groups[0]["lr"].mul_(0.5)
            p.grad = _gradient(p, s)
            opt.step()

    p, opt = make()
    train(p, opt, 0)
    buf, start = io.BytesIO(), p.detach().clone()
    torch.save(opt.state_dict(), buf)
    train(p, opt, 2)
    for where in ("cuda", "cpu"):
        buf.seek(0)
        q, again = make()
        q.data.copy_(start)
        again.load_state_dict(torch.load(buf, map_location=where))
        train(q, again, 2)
        assert torch.equal(p, q) and again.param_groups[0]["lr"].item() == opt.param_groups[0]["lr"].item()


@pytest.mark.parametrize("n", [6_000_077, 40_000_077])     # two and more state blocks a warp, and the most
@pytest.mark.parametrize("rounding", ["rn", "sr"])
@pytest.mark.parametrize("dtype,offset", [(torch.float32, 0), (torch.float32, 1), (torch.bfloat16, 0), (torch.bfloat16, 3)])
def test_windows_of_long_tensors_match_the_oracle(metis_lib, n, rounding, dtype, offset):
    """Windows at the start, across the borders of chunks and of the stretches that a warp takes, and at the ragged
    end; gradients that differ by orders of magnitude from a state block to the next, and whose pattern moves with the
    step, so that a block with its neighbour's exponent would show."""
    from spectral_quantized_gemm_b200.optim import AdamW
    g = torch.Generator(device="cuda").manual_seed(5)
    p = torch.nn.Parameter(torch.randn(n + offset, device="cuda", generator=g).to(dtype)[offset:])
    opt = AdamW([p], state_bits=8, rounding=rounding, seed=21, **HYPER)
    rng = np.random.default_rng(n)
    starts = [0, n // 128 * 128 - 1024, *(int(c) * 1024 - 1024 for c in rng.integers(1, n // 1024, 12)),
              *(int(c) * 16384 - 1024 for c in rng.integers(1, n // 16384, 8))]
    windows = [(a, min(a + 2048, n)) for a in starts]
    states = [tuple((np.zeros(b - a, np.uint8), np.zeros(-(-(b - a) // 128), np.uint8)) for _ in range(2)) for a, b in windows]
    block = torch.arange(n, device="cuda") // 128
    (b1, b2), lr, eps, wd = HYPER["betas"], HYPER["lr"], HYPER["eps"], HYPER["weight_decay"]
    for t in (1, 2, 3):
        scale = 10.0 ** -((block * 5 + t) % 9).float()
        p.grad = torch.empty(n + offset, dtype=dtype, device="cuda")[offset:].copy_(scale * torch.randn(n, device="cuda", generator=g))
        before = [_np(p[a:b]) for a, b in windows]
        opt.step()
        s = opt.state[p]
        for i, (a, b) in enumerate(windows):
            grad = _np(p.grad[a:b])
            m0, v0 = adamw.decode(*states[i][0], True), adamw.decode(*states[i][1], False)
            m, v = adamw.moments(m0, v0, grad, b1, b2)
            w = None
            if rounding == "sr":
                w = adamw.philox.stream_words(21, adamw.philox.tag(0, 4, 0), t, np.arange(a // 4, -(-b // 4), dtype=np.uint64))
                w = w.reshape(-1)[:b - a]
            new = (adamw.encode(m, True, None if w is None else w & np.uint64(0xFFFF)),
                   adamw.encode(v, False, None if w is None else w >> np.uint64(16)))
            for key, (codes, exponents) in zip(("exp_avg", "exp_avg_sq"), new):
                assert np.array_equal(s[key][a:b].cpu().numpy(), codes), (t, a, key)
                assert np.array_equal(s[key + "_exponent"][a // 128:-(-b // 128)].cpu().numpy(), exponents), (t, a, key)
            states[i] = new
            want = adamw.parameter(before[i], m, v, t, lr, b1, b2, eps, wd)
            size = lr / (1 - b1 ** t) * (np.abs(b1 * m0) + np.abs((1 - b1) * grad)) / (np.sqrt(v) / math.sqrt(1 - b2 ** t) + eps)
            bound = 3 * U * np.abs(before[i]) + 20 * U * size + 2.0 ** -148
            if dtype == torch.bfloat16:
                bound = bound + (2.0 ** -8 if rounding == "rn" else 2.0 ** -7) * (np.abs(want) + bound)
            assert np.all(np.abs(_np(p[a:b]) - want) <= bound), (t, a)
