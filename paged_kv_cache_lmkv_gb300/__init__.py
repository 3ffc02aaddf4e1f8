"""GB300-native batched paged-KV chunk gather / scatter (LMCache's store / retrieve
data path): a C-ABI CUDA library (include/lmkv.h, csrc/) and its Python binding."""
from . import lmkv  # noqa: F401
from .lmkv import (CachegenCodec, Offload, Pool, Rotary, LmkvError, append_layer,  # noqa: F401
                   attend_layer, attend_workspace_bytes, check, count_chunks, evict_layer,
                   scatter_chunks_shifted, scatter_layer_shifted, weigh_layer,
                   decode_store_ranges, enumerate_chunks,
                   gather_chunks, gather_chunks_fp8e4m3, gather_layer, pointer_array,
                   overlap_events, retrieve_layers, retrieve_layers_overlapped,
                   retrieve_layers_staged, scatter_chunks,
                   scatter_chunks_fp8e4m3, scatter_layer, staging_bytes, store_layers,
                   store_layers_overlapped, store_layers_staged, append_layer_normed,
                   attend_layer_window, attend_window_workspace_bytes, compact_pages, copy_pages, fork_pages,
                   pages_workspace_bytes, resize_pages)

__all__ = ["lmkv", "CachegenCodec", "Offload", "Pool", "LmkvError", "check", "count_chunks", "decode_store_ranges",
           "enumerate_chunks",
           "gather_chunks", "scatter_chunks", "gather_layer", "scatter_layer",
           "gather_chunks_fp8e4m3", "scatter_chunks_fp8e4m3", "pointer_array",
           "store_layers", "retrieve_layers", "store_layers_staged",
           "retrieve_layers_staged", "staging_bytes", "store_layers_overlapped",
           "retrieve_layers_overlapped", "overlap_events", "Rotary", "append_layer",
           "scatter_chunks_shifted", "scatter_layer_shifted", "attend_layer",
           "attend_workspace_bytes", "weigh_layer", "evict_layer", "append_layer_normed",
           "attend_layer_window", "attend_window_workspace_bytes", "copy_pages", "fork_pages",
           "resize_pages", "compact_pages", "pages_workspace_bytes"]
