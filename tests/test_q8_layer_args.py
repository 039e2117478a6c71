"""DSMoEQ8 without a GPU: where its buffers come from (the library's calls replaced by recorders)."""
import pytest
import torch

import mixture_experts_layer_score_b200 as M
from mixture_experts_layer_score_b200 import binding as B

CFG = M.make_cfg(d_model=64, n_routed=4, top_k=2, d_ff=64, max_tokens=8)


@pytest.fixture
def calls(monkeypatch):
    """A DSMoEQ8 whose buffers are on the CPU and whose library calls are recorded."""
    seen = {"alloc": [], "rows": []}

    def empty(stream, device, shapes):
        out = [torch.empty(s, dtype=t) for s, t in shapes]
        seen["alloc"] += [stream] * len(out)
        return out

    monkeypatch.setattr(B, "_empty", empty, raising=False)
    monkeypatch.setattr(B, "dsmoe_q8_quantize", lambda h, R, C, x, q, s, stream=None: None)
    monkeypatch.setattr(B, "dsmoe_norm_q8", lambda *a: None)
    monkeypatch.setattr(B, "dsmoe_forward_q8", lambda h, T, x, xq, xs, *a: seen["rows"].append((xq, xs)))
    layer = M.DSMoEQ8.__new__(M.DSMoEQ8)
    layer.cfg, layer.device, layer.handle, layer.w, layer.q = CFG, 0, None, {}, {}
    layer.k_active, layer.range_flags, layer._weights = 2, M.DSMOE_RANGE_ADD_SHARED, M.DsmoeQ8Weights()
    seen["layer"] = layer
    return seen


def test_rows_are_kept_with_the_outputs(calls):
    """A second call with the same `out` writes the first call's 8-bit rows again; it does not let
    them go while the first call may still read them."""
    layer, x = calls["layer"], torch.zeros(3, 64, dtype=torch.bfloat16)
    out = layer.alloc_outputs(3)
    layer.forward(x, out=out, stream=5)
    layer.forward(x, out=out, stream=5)
    assert calls["rows"][0][0] is calls["rows"][1][0] is out["x_q"][0]
    assert calls["rows"][0][1] is calls["rows"][1][1] is out["x_q"][1]
    layer.forward(x[:2], out=layer.alloc_outputs(2) | {"x_q": out["x_q"]})  # of another length: new ones
    assert calls["rows"][2][0].shape == (2, 64) and calls["rows"][2][1].shape == (2, 4)
    mine = layer.alloc_rows(3)
    layer.forward(x, out=out, x_q=mine)
    assert calls["rows"][3][0] is mine[0] and out["x_q"][0] is calls["rows"][0][0]


@pytest.mark.parametrize("stream", [None, 5])
def test_buffers_are_allocated_for_the_stream(calls, stream):
    layer, x = calls["layer"], torch.zeros(3, 64, dtype=torch.bfloat16)
    layer.forward(x, stream=stream)
    layer.forward_norm(x, None, None, 1e-6, stream=stream)
    assert len(calls["alloc"]) == 9 + 11 and set(calls["alloc"]) == {stream}


# ------------------------------------------------------------------------ what is refused
d, F, N, KS = 192, 704, 6, 2
BIG = M.make_cfg(d_model=d, n_routed=N, top_k=2, d_ff=F, n_shared=KS, d_ff_shared=128, max_tokens=8)


def pair(E, n, k, **kw):
    return (torch.zeros(E, n, k, dtype=kw.get("values", torch.float8_e4m3fn)),
            torch.zeros(E, -(-n // 128), kw.get("cols", M.dsmoe_q8_scale_cols(k)), dtype=kw.get("scales", torch.uint8)))


def pairs(E=N):
    return dict(W_gate=pair(E, F, d), W_up=pair(E, F, d), W_down=pair(E, d, F), Ws_gate=pair(KS, 128, d),
                Ws_up=pair(KS, 128, d), Ws_down=pair(KS, d, 128))


@pytest.fixture
def handle(monkeypatch):
    """A handle of BIG that the binding knows and the library never sees; its tensors are on the CPU."""
    h = 0  # (a layer of it has nothing to destroy)
    monkeypatch.setattr(B, "dsmoe_create", lambda cfg, device=0: h)
    monkeypatch.setattr(B, "dsmoe_q8_quantize_weights", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("S", (), {"synchronize": lambda s: 0})())
    live = B._Live(-1, BIG)
    monkeypatch.setitem(B._handles, h, live)

    class Lib:  # stands for the library where a call would read the handle
        def dsmoe_forward_q8(self, *a):
            return 0

        def dsmoe_set_expert_range(self, *a):
            return 0

        def __getattr__(self, name):
            return getattr(real, name)

    real = B._lib
    monkeypatch.setattr(B, "_lib", Lib())
    return h


def refused(call, *words):
    with pytest.raises(M.DsmoeError) as e:
        call()
    assert e.value.status == M.DSMOE_ERR_INVALID_ARG and all(w in str(e.value) for w in words), str(e.value)


BAD = [  # one expert tensor, what it is given as, and words of the refusal
    ("W_gate", pair(N, F, d, scales=torch.float32), "W_gate scales", "float32"),
    ("W_up", pair(N, F, d, cols=-(-d // 128)), "W_up scales"),  # as many columns as blocks
    ("W_down", pair(N, d, F, cols=-(-F // 128)), "W_down scales"),
    ("W_down", pair(N, F, d), "W_down"),  # transposed
    ("W_down", pair(N - 1, d, F), "W_down"),
    ("W_gate", pair(N, F, d, values=torch.float16), "W_gate values", "float16"),
    ("W_up", (pair(N, F, d)[0][:, ::2], pair(N, F, d)[1]), "W_up values"),
    ("Ws_gate", pair(KS - 1, 128, d), "Ws_gate"),
    ("Ws_down", pair(KS, d, 256), "Ws_down"),
]


@pytest.mark.parametrize("name,bad,words", [(b[0], b[1], b[2:]) for b in BAD])
def test_weight_pairs_are_checked(handle, name, bad, words):
    refused(lambda: M.DSMoEQ8(BIG, pairs() | {name: bad}), *words)
    x = torch.zeros(1, d, dtype=torch.bfloat16)
    call = lambda w: M.dsmoe_forward_q8(handle, 1, x, x.to(torch.float8_e4m3fn), torch.zeros(4, dtype=torch.uint8),  # noqa: E731
                                        None, None, 16, None, w, 16, 16, 16, 16, 16, 16, None, None, 0)
    refused(lambda: call(pairs() | {name: bad}), *words)
    call(pairs())


def test_layer_takes_what_fits(handle):
    layer = M.DSMoEQ8(BIG, pairs())
    assert layer.experts == N and layer._weights.W_down_scales == layer.q["W_down"][1].data_ptr()
    bf16 = {k: v[0].to(torch.bfloat16) for k, v in pairs().items()}
    assert M.DSMoEQ8(BIG, bf16).experts == N
    for k, v in (("W_gate", bf16["W_down"]), ("W_up", bf16["W_up"][:, :64]), ("Ws_up", bf16["Ws_up"][:1])):
        refused(lambda: M.DSMoEQ8(BIG, bf16 | {k: v}), k)
    flat = {k: tuple(t.reshape(-1) for t in v) for k, v in pairs().items()}
    assert M.DSMoEQ8(BIG, flat).experts == N
    raw = M.DSMoEQ8(BIG, {k: (16, 32) for k in pairs()})  # addresses are taken as they are
    assert raw.experts is None and raw._weights.W_up == 16 and raw._weights.Ws_down_scales == 32
    no_shared = M.make_cfg(d_model=d, n_routed=N, top_k=2, d_ff=F, max_tokens=8)
    B._handles[handle].cfg = no_shared
    layer = M.DSMoEQ8(no_shared, pairs())  # (shared experts that the configuration does not have are not read)
    assert "Ws_up" not in layer.q and layer._weights.Ws_up is None


def test_experts_of_the_weights_and_of_the_range(handle):
    """Weights of a part of the experts need that range, and whole ones the whole."""
    x, x_q = torch.zeros(1, d, dtype=torch.bfloat16), pair(1, 1, d)
    out = dict.fromkeys(("h", "topk_idx", "gates", "counts", "f", "P"), 16) | {"P_sum": None, "scores": None}
    part = M.DSMoEQ8(BIG, pairs(4))
    refused(lambda: part.forward(x, out=out, x_q=x_q), "4 routed experts")
    refused(lambda: part.set_expert_range(0, 3), "4 routed experts")
    part.set_expert_range(2, 6)
    part.w = {"W_router": 16}
    part.forward(x, out=out, x_q=x_q, stream=7)
    refused(lambda: M.DSMoEQ8(BIG, pairs()).set_expert_range(2, 6), "6 routed experts")
    M.dsmoe_set_expert_range(handle, 0, 3, 1)  # also past the object
    refused(lambda: part.forward(x, out=out, x_q=x_q, stream=7), "4 routed experts")


def test_forward_tensors_are_checked(handle):
    T = 3
    f32 = lambda *s: torch.zeros(s)  # noqa: E731
    ok = dict(x=torch.zeros(T, d, dtype=torch.bfloat16), x_q=pair(1, T, d)[0], x_scales=torch.zeros(T, 4, dtype=torch.uint8),
              residual=None, token_ids=None, W_router=torch.zeros(N, d, dtype=torch.bfloat16), b=f32(N), weights=pairs(),
              h=torch.zeros(T, d, dtype=torch.bfloat16), topk_idx=torch.zeros(T, 2, dtype=torch.int32), gates=f32(T, 2),
              counts=torch.zeros(N, dtype=torch.int32), f=f32(N), P=f32(N), P_sum=f32(N), scores_dbg=f32(T, N))
    call = lambda **kw: M.dsmoe_forward_q8(handle, T, *(ok | kw).values(), 0)  # noqa: E731
    call()
    call(h=torch.zeros(T + 1, d, dtype=torch.bfloat16), gates=f32(9, 2))  # outputs of a larger batch
    for name, bad in (("h", f32(T, d)), ("h", ok["h"][:2]), ("topk_idx", ok["topk_idx"].long()), ("gates", f32(T, 1)),
                      ("counts", f32(N)), ("f", f32(N - 1)), ("P", f32(N).double()), ("scores_dbg", f32(T, N - 1)),
                      ("W_router", f32(N, d)), ("W_router", ok["W_router"][1:]), ("b", f32(N - 1)),
                      ("token_ids", torch.zeros(T, dtype=torch.int64)), ("gates", f32(2, T).T), ("x_scales", f32(T))):
        refused(lambda: call(**{name: bad}), name)
    M.dsmoe_set_expert_range(handle, 0, N, M.DSMOE_RANGE_PARTIAL)
    refused(lambda: call(), "h ")
    call(h=f32(T, d))


@pytest.mark.parametrize("E", [1, 2])
@pytest.mark.parametrize("at", [2, 17])
def test_offsets_that_are_not_aligned_are_refused(E, at):
    buf = torch.zeros(1 << 13, dtype=torch.uint8)  # a handle of which only the configuration is looked at
    for call in (lambda: M.dsmoe_q8_matmul(buf.data_ptr(), E, 1, 8, 16, at, *[16] * 5, 0),
                 lambda: M.dsmoe_q8_gated_matmul(buf.data_ptr(), E, 1, 16, 16, at, *[16] * 8, 0)):
        refused(call, "offsets", "aligned")
