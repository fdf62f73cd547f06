"""liblla: causal Local Linear Attention forward for GB300 (sm_103a).

The compute path is the C-ABI shared library ``liblla.so`` (built from ``csrc/``); the Python
module ``binding`` marshals torch tensors into its entry points. Importing this package does not
load the library: the binding is loaded on first use and raises if the library is missing.
"""
from . import workloads  # noqa: F401

_BINDING = {
    "lla_forward", "lla_forward_ws", "lla_workspace_size", "lla_moments", "lla_forward_host",
    "lla_stream_status", "lla_status_string", "lla_version", "LlaError", "library_path",
    "launch_count", "profile_enable", "profile_collect", "lla_forward_noalloc",
    "lla_parallax_forward", "lla_decode", "lla_parallax_decode", "lla_parallax_backward",
    "Options", "PagedCache", "lla_paged_append", "lla_paged_attention", "lla_paged_workspace_size",
    "lla_paged_evict", "lla_paged_tree_attention", "lla_paged_tree_workspace_size",
    "RotarySpec", "ROTARY_HALVES", "ROTARY_INTERLEAVED", "STRETCH_NONE", "STRETCH_POSITIONS", "STRETCH_BASE",
    "STRETCH_WAVELENGTHS", "lla_rotary", "lla_paged_append_rotary", "lla_paged_fork", "lla_paged_free", "lla_paged_grow",
    "lla_paged_copy", "lla_paged_compact",
}


def __getattr__(name):
    if name in _BINDING:
        from . import binding
        globals()[name] = getattr(binding, name)  # found without this function from now on
        return globals()[name]
    raise AttributeError(name)
