"""Refusals of the 8-bit path's entry points that need no GPU: arguments are checked before
anything is launched."""
import ctypes

import pytest
import torch

import mixture_experts_layer_score_b200 as M


def test_scale_cols():
    assert [M.dsmoe_q8_scale_cols(c) for c in (-1, 0, 1, 128, 512, 513, 7168)] == [0, 0, 4, 4, 4, 8, 56]


@pytest.mark.parametrize("call", [
    lambda: M.dsmoe_q8_quantize(None, 1, 16, 16, 16, 16, 0),
    lambda: M.dsmoe_q8_quantize_weights(None, 1, 1, 16, 16, 16, 16, 0),
    lambda: M.dsmoe_norm_q8(None, 1, 16, None, 16, 1e-6, None, 16, None, None, 0),
    lambda: M.dsmoe_norm_backward(None, 1, 16, None, 16, 16, 1e-6, 16, 16, 0),
    lambda: M.dsmoe_q8_matmul(None, 1, 1, 8, 16, 16, 16, 16, 16, 16, 16, 0),
    lambda: M.dsmoe_q8_gated_matmul(None, 1, 1, 16, 16, 16, 16, 16, 16, 16, 16, 16, 16, 16, 0),
    lambda: M.dsmoe_forward_q8(None, 1, 16, 16, 16, None, None, 16, None, M.DsmoeQ8Weights(), 16, 16, 16, 16, 16, 16,
                               None, None, 0),
])
def test_a_null_handle_is_refused(call):
    with pytest.raises(M.DsmoeError) as e:
        call()
    assert e.value.status == M.DSMOE_ERR_INVALID_ARG


def test_tensors_of_another_kind_are_refused():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    for bad in (dict(x=x.float()), dict(x=x[:2]), dict(q=q.int()), dict(s=s[:, :2].contiguous()),
                dict(x=torch.zeros(32, 4, dtype=torch.bfloat16).T), dict()):  # the last: tensors on the CPU
        a = dict(x=x, q=q, s=s) | bad
        with pytest.raises(M.DsmoeError) as e:
            M.dsmoe_q8_quantize(None, 4, 32, a["x"], a["q"], a["s"], 0)
        assert e.value.status == M.DSMOE_ERR_INVALID_ARG


class TestHandle:
    """Sizes and pointers, with a handle that no check looks into deeper than its configuration."""

    @pytest.fixture(autouse=True)
    def fake(self):
        # a dsmoe_handle starts with its dsmoe_cfg; the checks below read nothing else
        self.buf = ctypes.create_string_buffer(1 << 16)
        cfg = M.make_cfg(d_model=64, n_routed=1, top_k=1, d_ff=64, max_tokens=8)
        ctypes.memmove(self.buf, ctypes.byref(cfg), ctypes.sizeof(cfg))
        self.h = ctypes.addressof(self.buf)

    def status(self, call):
        with pytest.raises(M.DsmoeError) as e:
            call()
        return e.value.status

    @pytest.mark.parametrize("R,C,expect", [(-1, 16, 1), (1, 0, 1), (1, 24, 2), (1, 32784, 2), (1 << 31, 16, 2)])
    def test_quantize_sizes(self, R, C, expect):
        assert self.status(lambda: M.dsmoe_q8_quantize(self.h, R, C, 16, 16, 16, 0)) == expect

    @pytest.mark.parametrize("x,q,s", [(None, 16, 16), (16, None, 16), (16, 16, None), (8, 16, 16), (16, 24, 16),
                                       (16, 16, 6)])
    def test_quantize_pointers(self, x, q, s):
        assert self.status(lambda: M.dsmoe_q8_quantize(self.h, 1, 16, x, q, s, 0)) == 1

    @pytest.mark.parametrize("E,N,K,expect", [(0, 1, 16, 1), (1, 0, 16, 1), (513, 1, 16, 2), (1, 32769, 16, 2),
                                              (1, 1, 8, 2)])
    def test_quantize_weights_sizes(self, E, N, K, expect):
        assert self.status(lambda: M.dsmoe_q8_quantize_weights(self.h, E, N, K, 16, 16, 16, 0)) == expect

    def test_norm(self):
        ok = dict(T=1, x=16, res=None, w=16, eps=1e-6, r=None, u=16, q=None, s=None)
        for bad, expect in ((dict(T=-1), 1), (dict(T=9), 3), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
                            (dict(eps=float("inf")), 1), (dict(q=16), 1), (dict(s=16), 1), (dict(u=None), 1),
                            (dict(x=None), 1), (dict(w=None), 1), (dict(x=8), 1), (dict(res=8), 1), (dict(u=8), 1),
                            (dict(q=8, s=16), 1), (dict(q=16, s=18), 1)):
            a = ok | bad
            assert self.status(lambda: M.dsmoe_norm_q8(self.h, a["T"], a["x"], a["res"], a["w"], a["eps"], a["r"],
                                                       a["u"], a["q"], a["s"], 0)) == expect, bad

    def test_norm_backward(self):
        ok = dict(T=1, dy=16, dres=None, r=16, w=16, eps=1e-6, dx=16, dw=16)
        for bad, expect in ((dict(T=-1), 1), (dict(T=9), 3), (dict(eps=-1.0), 1), (dict(dy=None), 1),
                            (dict(r=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(dres=8), 1),
                            (dict(dw=8), 1), (dict(T=0, dw=None), 1)):
            a = ok | bad
            assert self.status(lambda: M.dsmoe_norm_backward(self.h, a["T"], a["dy"], a["dres"], a["r"], a["w"],
                                                             a["eps"], a["dx"], a["dw"], 0)) == expect, bad

    @pytest.mark.parametrize("E,R,N,K,expect", [(0, 1, 8, 16, 1), (1, -1, 8, 16, 1), (1, 1, 0, 16, 1),
                                                (1, 1, 12, 16, 2), (1, 1, 8, 8, 2), (1, 1, 32776, 16, 2),
                                                (1, 1, 8, 32784, 2),
                                                (513, 1, 8, 16, 2), (1, 1 << 31, 8, 16, 2)])
    def test_product_sizes(self, E, R, N, K, expect):
        p = [16] * 6
        assert self.status(lambda: M.dsmoe_q8_matmul(self.h, E, R, N, K, *p, 0)) == expect
        if N != 8:
            return
        p = [16] * 9
        assert self.status(lambda: M.dsmoe_q8_gated_matmul(self.h, E, R, 16, K, *p, 0)) == expect
        assert self.status(lambda: M.dsmoe_q8_gated_matmul(self.h, 1, 1, 8, 16, *p, 0)) == 2

    def test_product_pointers(self):
        for i in range(6):
            for bad in ((None, 6) if i else (None,)):  # (offsets may only be NULL where E is 1)
                p = [16] * 6
                p[i] = bad
                assert self.status(lambda: M.dsmoe_q8_matmul(self.h, 2, 1, 8, 16, *p, 0)) == 1
        for i in range(9):
            for bad in ((None, 6) if i else (None,)):
                p = [16] * 9
                p[i] = bad
                assert self.status(lambda: M.dsmoe_q8_gated_matmul(self.h, 2, 1, 16, 16, *p, 0)) == 1
        for i in (1, 3, 5):  # values need 16 bytes
            p = [16] * 6
            p[i] = 8
            assert self.status(lambda: M.dsmoe_q8_matmul(self.h, 2, 1, 8, 16, *p, 0)) == 1
