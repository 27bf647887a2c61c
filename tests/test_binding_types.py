"""The binding of the tree, window and page calls refuses tensors of another type than the call's, of the same element
size too (a float16 cache for bf16, floats for lengths), on CPU: tensors and library are stand-ins."""
import numpy as np
import pytest
import torch

import mla_latent_kv_24_b200 as mla

F, B, I, L, U = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint64


class Tensor:
    """What the binding asks of a CUDA tensor."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, dtype):
        self.dtype, self.itemsize = dtype, dtype.itemsize

    def get_device(self):
        return 0

    def numel(self):
        return 1 << 40

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256


class Lib:
    def __getattr__(self, name):
        return lambda *a: 0


@pytest.fixture(autouse=True)
def stand_ins(monkeypatch):
    mla._here()                                        # finds torch
    monkeypatch.setattr(mla, "_here", lambda: 0)
    monkeypatch.setattr(mla, "load", Lib)


H = np.ones(1, np.int32)
POOL = dict(seq_lens=I, page_table=I, batch=1, max_pages=1, page_refs=I, n_pages_total=1)
VIEW = dict(page_table=I, seq_lens=I, seq_lens_host=H, batch=1, max_pages=1, n_pages_total=1, workspace=torch.uint8)
WIN = dict(VIEW, s_q=1, sinks=1, window=1)
# a float tensor's type stands as "e": the call's
CALLS = {
    "mla_decode_tree": dict(VIEW, q="e", W_uk="e", W_uv="e", latent_cache="e", n_nodes=I, n_nodes_host=H, depths=I, tree_mask=L,
                            max_nodes=1, out="e"),
    "mla_decode_window": dict(WIN, q="e", W_uk="e", W_uv="e", latent_cache="e", out="e"),
    "gqla_decode_window": dict(WIN, q="e", expanded_cache="e", latent_cache="e", out="e"),
    "mla_cache_append_slots": dict(h="e", hidden=8, W_dkv="e", W_kr="e", req_idx=I, slots=I, positions=I, n_tok=1, page_table=I,
                                   batch=1, max_pages=1, n_pages_total=1, latent_cache="e"),
    "mla_cache_reserve": dict(POOL, new_lens=I),
    "mla_cache_fork": dict(POOL, src_req=I, dst_req=I, n_fork=1, latent_cache="e", expanded_cache="e", n_layers=1),
    "mla_cache_release": dict(POOL, req_idx=I, first_page=I, last_page=I, n_req=1),
    "mla_cache_accept": dict(POOL, ctx_lens=I, n_nodes=I, accepted=I, n_accepted=I, max_nodes=1, latent_cache="e",
                             expanded_cache="e", n_layers=1),
}
OTHERS = {B: (torch.float16, torch.int16, torch.uint16, F), F: (I, torch.uint32, torch.float64, B), I: (F, torch.uint32, L),
          L: (torch.float64, I), torch.uint8: ()}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", CALLS)
def test_types(name, dtype):
    e = B if dtype == "bf16" else F
    types = {k: e if isinstance(v, str) else v for k, v in CALLS[name].items()}
    d, fn = mla.make_dims(dtype=dtype), getattr(mla, name)

    def call(**changed):
        args = {k: Tensor(v) if isinstance(v, torch.dtype) else v for k, v in dict(types, **changed).items()}
        fn(d, stream=0, **args)

    call()
    for arg, t in types.items():
        if isinstance(t, torch.dtype):
            for wrong in OTHERS[t]:
                with pytest.raises(ValueError, match=arg):
                    call(**{arg: wrong})


def test_masks_may_be_signed_or_not():
    types = {k: B if isinstance(v, str) else v for k, v in CALLS["mla_decode_tree"].items()}
    for t in (L, U):
        mla.mla_decode_tree(mla.make_dims(), stream=0, **{k: Tensor(v) if isinstance(v, torch.dtype) else v
                                                          for k, v in dict(types, tree_mask=t).items()})
