"""Per-head latent-KV decode on B200 (sm_100a): a C-ABI CUDA library plus thin
torch wrappers.  See include/lk.h (the latent path) and include/lk_serving.h
(the serving operators beside it) for the boundary.

The library (liblk.so) is loaded on first use of a wrapper, so the input
generators (``synth``, ``configs``) import without it; every wrapper still
fails loudly when the library is missing."""
import importlib

_API = ("LatentCache", "LowrankWeight", "device_status", "latent_decode_attn", "latent_decode_step",
        "latent_project_append", "lowrank_linear", "quantize_latent", "quantize_rows_i8", "rmsnorm_quant_i8",
        "rmsnorm_hadamard_quant_i8", "swiglu_quant_i8", "workspaces", "kernel_launches", "dense_decode_attn", "reconstruct_kv",
        "rope_table", "latent_decode_attn_rope", "OutsplitFfn")

_SERVING = ("PagedKVCache", "paged_append", "paged_decode_attn", "paged_evict", "W4Weight", "w4_linear",
            "rmsnorm_gate_residual")


def __getattr__(name):
    if name in _SERVING:
        value = getattr(importlib.import_module(".serving", __name__), name)
        globals()[name] = value  # found at once from now on: this look-up costs a microsecond a call
        return value
    if name in _API:
        return getattr(importlib.import_module(".api", __name__), name)
    if name == "LkError":
        return importlib.import_module("._lib", __name__).LkError
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


__all__ = list(_API) + list(_SERVING) + ["LkError"]
