"""B200-native (sm_100a) Fast-weight Product Key Memory: the chunked
read-then-write memory step behind a C ABI (include/fwpkm.h), and the paged
key-value cache of the attention layers beside it (include/fwpkm_cache.h).

    from sparse_weight_memory_b200 import FwPKMState, KVCache
    mem = FwPKMState(N=256 * 256, dq=512, dv=512, topk=8, chunk=256)
    mem.set_tables(subkeys, values)
    out = mem.step(Q, Vtarget, gate, eta=1.0)       # torch CUDA tensors

    cache = KVCache(pages=1024, page_size=64, kv_heads=8, dim=128)
    q = cache.append(k, v, table, lengths, q=q, freqs=freqs)  # one token a sequence
    out = cache.attend(q, table, lengths)
"""
from .fwpkm import FwPKMState, FwpkmError, load_library, LIB_PATH  # noqa: F401

__all__ = ["FwPKMState", "FwpkmError", "KVCache", "load_library", "LIB_PATH"]


def __getattr__(name):  # torch is imported only where the cache is used
    if name == "KVCache":
        from .cache import KVCache
        return KVCache
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
