"""What the binding of the speculative-step calls takes by pointer: tensors of
another type, length, shape, layout or device than the kernels read are refused
before the library is called, and right ones reach it.  The library is a
recorder here and the context's device is the host (index -1)."""
import types

import pytest
import torch

from hybrid_sliding_window_gb300 import api

HQ, HKV, D, N, BS = 8, 2, 64, 6, 3
I64, I32, F32, BF = torch.int64, torch.int32, torch.float32, torch.bfloat16


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name in ("swa_tree_bytes", "swa_plan_bytes"):
                return 512
            self.calls.append((name, args))
            return api.SWA_OK
        return call


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(api, "lib", lambda: r)
    monkeypatch.setattr(api, "_stream", lambda s=None: None)
    return r


def ctx(io=BF):
    return types.SimpleNamespace(handle=None, gpu=-1, io_dtype=io, num_q_heads=HQ, head_dim=D,
                                 layers=[dict(kind=api.LAYER_FULL, num_kv_heads=HKV),
                                         dict(kind=api.LAYER_SLIDING, num_kv_heads=HKV)])


def z(*shape, t=I64):
    return torch.zeros(shape, dtype=t)


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 1


def elsewhere(*shape, t=I64):
    return torch.zeros(shape, dtype=t).as_subclass(Elsewhere)


GOOD = {
    "swa_tree_plan": lambda: dict(parents=z(N, t=I32), prefix_lens=z(BS), qo_indptr=z(BS + 1), n_tokens=N, max_new=4,
                                  tree=z(512, t=torch.uint8), positions=z(N)),
    "swa_attn_tree": lambda: dict(layer=1, req_to_token=z(4, 64, t=I32), req_idx=z(BS), prefix_lens=z(BS), qo_indptr=z(BS + 1),
                                  n_tokens=N, max_new=4, max_seq_len=60, plan=z(512, t=torch.uint8), tree=z(512, t=torch.uint8),
                                  q=z(N, HQ, D, t=BF), sinks=z(HQ, t=F32), sm_scale=0.1, out=z(N, HQ, D, t=BF),
                                  ws=z(64, t=torch.uint8)),
    "swa_qk_norm_rope_store": lambda: dict(layer=1, q=z(N, HQ, D, t=BF), k=z(N, HKV, D, t=BF), v=z(N, HKV, D, t=BF), positions=z(N),
                                           full_loc=z(N), q_out=z(N, HQ, D, t=BF), swa_loc=z(N), q_weight=z(D, t=F32),
                                           k_weight=z(D, t=F32), cos_sin=z(100, 32, t=F32), rot_dim=32),
    "swa_commit_tree": lambda: dict(req_to_token=z(4, 64, t=I32), req_idx=z(BS), prefix_lens=z(BS), accepted=z(BS, 5, t=I32),
                                    n_accepted=z(BS, t=I32)),
    "swa_copy_kv": lambda: dict(src=z(7), dst=z(7)),
}

BAD = {
    "swa_tree_plan": [("parents", z(N)), ("parents", z(N - 1, t=I32)), ("qo_indptr", z(BS)), ("prefix_lens", z(BS, t=I32)),
                      ("positions", z(N - 1)), ("positions", z(N, t=I32)), ("tree", elsewhere(512, t=torch.uint8)),
                      ("parents", z(2 * N, t=I32)[::2])],
    "swa_attn_tree": [("layer", 2), ("layer", -1), ("req_to_token", z(4, 64)), ("req_to_token", z(64, t=I32)),
                      ("req_to_token", z(4, 128, t=I32)[:, :64]), ("req_idx", z(BS - 1)), ("qo_indptr", z(BS)),
                      ("plan", z(511, t=torch.uint8)), ("tree", z(511, t=torch.uint8)), ("q", z(N, HQ, D, t=F32)),
                      ("q", z(N - 1, HQ, D, t=BF)), ("q", z(N, 2 * HQ, D, t=BF)[:, :HQ]), ("out", z(N, HQ, D, t=torch.half)),
                      ("out", z(N, HQ, D // 2, t=BF)), ("sinks", z(HQ, t=BF)), ("sinks", z(HQ - 1, t=F32)),
                      ("sinks", z(HQ + 1, t=F32)), ("ws", elsewhere(64, t=torch.uint8)), ("q", elsewhere(N, HQ, D, t=BF))],
    "swa_qk_norm_rope_store": [("layer", 5), ("q_weight", z(D, t=BF)), ("q_weight", z(D - 1, t=F32)), ("k_weight", z(HKV * D, t=F32)),
                               ("k_weight", z(2 * D, t=F32)[::2]), ("cos_sin", z(100, 32, t=BF)), ("cos_sin", z(100, 64, t=F32)),
                               ("cos_sin", z(3200, t=F32)), ("cos_sin", z(100, 64, t=F32)[:, :32]), ("positions", z(N - 1)),
                               ("positions", z(N, t=I32)), ("full_loc", z(N - 1)), ("full_loc", z(N, t=I32)), ("swa_loc", z(N - 2)),
                               ("q", z(N, HQ, D, t=F32)), ("q", z(N, HQ + 1, D, t=BF)), ("q", z(N, HQ, 2 * D, t=BF)),
                               ("q", z(N, HQ * D, t=BF)), ("q", z(N, HQ, 2 * D, t=BF)[:, :, ::2]),
                               ("q", z(N, 2 * HQ, D, t=BF)[:, ::2]), ("k", z(N, HKV + 1, D, t=BF)), ("v", z(N - 1, HKV, D, t=BF)),
                               ("k", z(N + 1, HKV, D, t=BF)), ("q_out", z(N, HQ, D, t=F32)), ("q_out", z(N - 1, HQ, D, t=BF)),
                               ("v", elsewhere(N, HKV, D, t=BF))],
    "swa_commit_tree": [("req_to_token", z(4, 64)), ("req_idx", z(BS - 1)), ("accepted", z(BS, 5)), ("accepted", z(BS * 5, t=I32)),
                        ("accepted", z(BS - 1, 5, t=I32)), ("accepted", z(BS, 10, t=I32)[:, :5]), ("n_accepted", z(BS)),
                        ("n_accepted", z(BS - 1, t=I32))],
    "swa_copy_kv": [("src", z(6)), ("src", z(7, t=I32)), ("dst", z(7, t=I32)), ("dst", z(14)[::2]), ("dst", elsewhere(7))],
}


@pytest.mark.parametrize("name", list(GOOD))
def test_right_arguments_reach_the_library(rec, name):
    args = GOOD[name]()
    getattr(api, name)(ctx(), **args)
    assert [c[0] for c in rec.calls] == [name]
    given = rec.calls[0][1]
    for key, t in args.items():
        if isinstance(t, torch.Tensor):
            assert t.data_ptr() in given, key


@pytest.mark.parametrize("name,key,value", [(n, k, v) for n in BAD for k, v in BAD[n]],
                         ids=[f"{n}-{k}-{i}" for n in BAD for i, (k, _) in enumerate(BAD[n])])
def test_wrong_arguments_are_refused(rec, name, key, value):
    with pytest.raises(api.SwaError) as e:
        getattr(api, name)(ctx(), **{**GOOD[name](), key: value})
    assert e.value.status == api.SWA_ERR_INVALID and not rec.calls


def test_what_a_call_does_not_read_is_not_looked_at(rec):
    q, k, v, out = z(N, HQ, D, t=BF), z(N, HKV, D, t=BF), z(N, HKV, D, t=BF), z(N, HQ, D, t=BF)
    # no rotation, a full layer, queries only
    api.swa_qk_norm_rope_store(ctx(), 0, q, k, v, z(1, t=I32), z(N), out, swa_loc=z(1, t=I32), cos_sin=z(3, t=BF))
    api.swa_qk_norm_rope_store(ctx(), 1, q, None, None, None, z(2, t=I32), out, swa_loc=z(1))
    assert [c[1][9] for c in rec.calls] == [None, None] and [c[1][18] for c in rec.calls] == [None, None]
    # byte buffers of any type; a full layer's plan of any size
    args = {**GOOD["swa_attn_tree"](), "plan": z(64), "tree": z(64), "ws": z(8, t=F32)}
    api.swa_attn_tree(ctx(), **args)
    assert rec.calls[-1][1][-2] == 32
    api.swa_attn_tree(ctx(), **{**args, "layer": 0, "plan": z(1, t=I32)})
    api.swa_attn_tree(ctx(), **{**args, "layer": 0, "plan": None})


def test_slices_of_a_fused_projection_and_absent_parts(rec):
    qkv = z(N, HQ + 2 * HKV, D, t=BF)
    q, k, v = qkv.split([HQ, HKV, HKV], 1)
    api.swa_qk_norm_rope_store(ctx(), 0, q, k, v, None, z(N), z(N, HQ, D, t=BF))
    api.swa_qk_norm_rope_store(ctx(), 0, None, k, v, None, z(N), None)
    api.swa_qk_norm_rope_store(ctx(), 0, q, None, None, None, None, z(N, HQ, D, t=BF))
    stride = (HQ + 2 * HKV) * D
    assert [c[1][3] for c in rec.calls] == [stride, 0, stride] and [c[1][5] for c in rec.calls] == [stride, stride, 0]
    with pytest.raises(api.SwaError):
        api.swa_qk_norm_rope_store(ctx(), 0, None, None, None, None, None, None)
