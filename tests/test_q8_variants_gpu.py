"""Every variant of the 8-bit product kernel (tests/q8_cases.py) against the float64 product of the
same operands, its bounded waits running out, and all of them in flight together."""
import pytest
import torch

import mixture_experts_layer_score_b200 as M
from tests import q8_cases as C
from tests.q8_cases import E8, F8, F64, values

pytestmark = pytest.mark.gpu
FIRST, BEHIND = 3, 5  # rows before the first group and behind the last


@pytest.fixture(scope="module")
def handle():
    h = M.dsmoe_create(M.make_cfg(d_model=64, n_routed=1, top_k=1, d_ff=64, max_tokens=1))
    yield h
    assert M.dsmoe_get_status(h) == M.DSMOE_OK
    M.dsmoe_destroy(h)


def empty8(*shape):
    return (torch.empty(shape, dtype=F8, device="cuda"),
            torch.empty((*shape[:-2], -(-shape[-2] // 128) if len(shape) == 3 else shape[-2],
                         M.dsmoe_q8_scale_cols(shape[-1])), dtype=E8, device="cuda"))


class Case:
    """Operands of a grouped product, its call and its check."""

    def __init__(self, handle, output, counts, N, K, seed=0, first=FIRST, behind=BEHIND):
        self.output, self.N, self.K, self.E = output, N, K, len(counts)
        self.R = first + sum(counts) + behind
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(self.R, K, generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(self.R, 1, generator=g, device="cuda"))
        self.a = empty8(self.R, K)
        M.dsmoe_q8_quantize(handle, self.R, K, x.bfloat16(), *self.a)
        self.w = []
        for _ in range(2 if output == C.GATED else 1):
            W = torch.empty(self.E, N, K, dtype=torch.bfloat16, device="cuda").normal_(0, K ** -0.5, generator=g)
            W *= torch.exp2(torch.arange(N, device="cuda") % 3 - 1).bfloat16()[:, None]
            self.w.append(empty8(self.E, N, K))
            M.dsmoe_q8_quantize_weights(handle, self.E, N, K, W, *self.w[-1])
        ends = [first]
        for c in counts:
            ends.append(ends[-1] + c)
        self.ends, self.off = ends, torch.tensor(ends, dtype=torch.int32, device="cuda")

    def outputs(self):
        if self.output == C.BF16:
            return [torch.full((self.R, self.N), 7.0, dtype=torch.bfloat16, device="cuda")]
        out = empty8(self.R, self.N)
        for t in out:
            t.view(torch.uint8).fill_(9)
        return list(out)

    def call(self, handle, out, stream=None):
        args = (handle, self.E, self.R, self.N, self.K, self.off, *self.a)
        if self.output == C.BF16:
            M.dsmoe_q8_matmul(*args, *self.w[0], *out, stream)
        else:
            M.dsmoe_q8_gated_matmul(*args, *self.w[0], *self.w[1], *out, stream)

    def check(self, out):
        outside = torch.ones(self.R, dtype=torch.bool, device="cuda")
        outside[self.ends[0]:self.ends[-1]] = False
        for t in out:
            assert bool((t[outside] == 7).all() if self.output == C.BF16 else (t.view(torch.uint8)[outside] == 9).all())
        for e in range(self.E):
            rows = slice(self.ends[e], self.ends[e + 1])
            if rows.start == rows.stop:
                continue
            a = values(self.a[0][rows], self.a[1][rows])
            w = [values(q[e], s[e]) for q, s in self.w]
            (C.check_plain if self.output == C.BF16 else C.check_gated)(a, *w, *(t[rows] for t in out))


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("output,variant,counts,N,K", C.GROUPED)
def test_grouped(handle, output, variant, counts, N, K):
    assert C.variant(output, len(counts), FIRST + sum(counts) + BEHIND, N, K, sms()) == variant
    case = Case(handle, output, counts, N, K)
    out, again = case.outputs(), case.outputs()
    case.call(handle, out)
    case.check(out)
    case.call(handle, again)
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(out, again))


@pytest.mark.parametrize("variant,T,d,Fs,shared", C.SHARED)
def test_shared_experts(variant, T, d, Fs, shared):
    """The fp32 product: what the layer's shared experts leave in the workspace, the base (bf16) plus the
    experts' rows one after another."""
    assert C.variant(C.FP32, 1, T, d, Fs, sms()) == variant
    cfg = M.make_cfg(d_model=d, n_routed=4, top_k=1, d_ff=64, n_shared=shared, d_ff_shared=Fs, max_tokens=T)
    g = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(0, s[-1] ** -0.5, generator=g)  # noqa: E731
    w = dict(W_gate=draw(4, 64, d), W_up=draw(4, 64, d), W_down=draw(4, d, 64), W_router=draw(4, d),
             Ws_gate=draw(shared, Fs, d), Ws_up=draw(shared, Fs, d), Ws_down=draw(shared, d, Fs))
    layer = M.DSMoEQ8(cfg, w)
    x = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    base = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    layer.forward(x, residual=base)
    torch.cuda.synchronize()
    assert M.dsmoe_get_status(layer.handle) == M.DSMOE_OK
    got = M.workspace_view(layer.handle, "Hs")[:T].to(F64)
    m = M.workspace_view(layer.handle, "A1s").reshape(-1).view(torch.uint8)  # the last expert's 8-bit rows
    S = M.dsmoe_q8_scale_cols(Fs)
    last = values(m[:T * Fs].view(T, Fs).view(F8), m[T * Fs:T * (Fs + S)].view(T, S).view(E8))
    a = values(*(lambda q: (M.dsmoe_q8_quantize(layer.handle, T, d, x, *q), q)[1])(empty8(T, d)))
    want, err = base.to(F64), 2.0 ** -23 * base.to(F64).abs()
    for i in range(shared):
        wd = values(layer.q["Ws_down"][0][i], layer.q["Ws_down"][1][i])
        if i == shared - 1:
            rows, slack = last, 0.0
        else:  # an expert before the last: its rows are not kept; theirs within half an e4m3 step
            y = [a @ values(layer.q[n][0][i], layer.q[n][1][i]).T for n in ("Ws_gate", "Ws_up")]
            rows = y[0] / (1 + torch.exp(-y[0])) * y[1]
            step = rows.abs().unflatten(1, (-1, 128 if Fs % 128 == 0 else 64)).amax(2)
            slack = 2.0 ** -4 * (1 + 2.0 ** -4) * rows.abs() + 2.0 ** -17 * step.repeat_interleave(Fs // step.shape[1], 1)
            slack = slack @ wd.abs().T
        mag = rows.abs() @ wd.abs().T
        want = want + rows @ wd.T
        err = err + (Fs + 2 + shared) * 2.0 ** -23 * mag + slack
    assert bool(((got - want).abs() <= err + 2.0 ** -23 * want.abs()).all())
    layer.close()


# ------------------------------------------------------------- bounded waits, two at once
WAITS = [i for i, c in enumerate(C.GROUPED) if c[1] in ((32, False, False), (112, False, False), (240, False, False),
                                                       (160, False, True), (32, False, True), (112, False, True),
                                                       (112, True, False), (32, True, True))]


@pytest.mark.parametrize("i", WAITS)
def test_wait_limit_runs_out(i):
    """With a limit of 1 ns some role gives up, the kernel drains what it started and returns, the
    status says so once; with the default limit the same handle's product is right again."""
    output, variant, counts, N, K = C.GROUPED[i]
    h = M.dsmoe_create(M.make_cfg(d_model=64, n_routed=1, top_k=1, d_ff=64, max_tokens=1))
    case = Case(h, output, counts, N, K)
    torch.cuda.synchronize()
    M.dsmoe_set_wait_limit(h, 1)
    case.call(h, case.outputs())
    torch.cuda.synchronize()
    assert M.dsmoe_get_status(h) == M.DSMOE_ERR_DEVICE_TIMEOUT
    assert M.dsmoe_get_status(h) == M.DSMOE_OK
    M.dsmoe_set_wait_limit(h, 2_000_000_000)
    out = case.outputs()
    case.call(h, out)
    case.check(out)
    assert M.dsmoe_get_status(h) == M.DSMOE_OK
    M.dsmoe_destroy(h)


def test_variants_in_flight_together():
    """Every variant on a stream of its own, all in flight, give the bits of each alone."""
    runs = []
    for i, (output, variant, counts, N, K) in enumerate(C.GROUPED):
        h = M.dsmoe_create(M.make_cfg(d_model=64, n_routed=1, top_k=1, d_ff=64, max_tokens=1))
        case = Case(h, output, counts, N, K, seed=i)
        out = [case.outputs(), case.outputs()]
        case.call(h, out[0])
        runs.append((h, case, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for h, case, out, stream in runs:
            case.call(h, out[1], stream)
    torch.cuda.synchronize()
    for h, case, out, stream in runs:
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(*out))
        assert M.dsmoe_get_status(h) == M.DSMOE_OK
        M.dsmoe_destroy(h)
