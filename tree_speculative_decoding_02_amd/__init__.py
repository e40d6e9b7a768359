"""MI355X (gfx950) Bole tree verification and accepted-path commit for linear-recurrence
layers. The compute lives in libbole.so (HIP kernels behind the C ABI of include/bole.h);
``bole`` is its thin Python binding."""
from .bole import (bind_build_tree, bole_build_tree, bind_tree_accept, bole_tree_accept, bind_commit_path, bind_commit_path_layers, bind_tree_verify,
                   bind_tree_verify_lazy_commit, bind_tree_verify_lazy_commit_layers,
                   bind_tree_verify_layers, bole_commit_path, bole_commit_path_layers,
                   bole_tree_prepare, bole_tree_verify, bole_tree_verify_lazy_commit,
                   bole_tree_verify_lazy_commit_layers, bole_tree_verify_layers,
                   bole_tree_verify_naive, BoleError, MAX_TREE_NODES)
from .delta import (bind_delta_commit_path, bind_delta_prefill, bind_delta_step,
                    bind_delta_tree_verify, bole_delta_commit_path, bole_delta_prefill,
                    bole_delta_prefill_workspace_size, bole_delta_step, bole_delta_tree_verify)
from .window import (bind_window_attention, bole_window_attention,
                     bole_window_workspace_size)
from .linear import (bind_linear_prefill, bind_linear_step, bole_linear_prefill,
                     bole_linear_prefill_workspace_size, bole_linear_step)
from .paged import (bind_cache_append, bind_prefix_attention, bind_qk_norm_rotary, bole_cache_append,
                    bole_prefix_attention, bole_prefix_workspace_size, bole_qk_norm_rotary)

__all__ = ["bind_linear_prefill", "bind_linear_step", "bole_linear_prefill",
           "bole_linear_prefill_workspace_size", "bole_linear_step",
           "bind_cache_append", "bind_prefix_attention", "bind_qk_norm_rotary", "bole_cache_append",
           "bole_prefix_attention", "bole_prefix_workspace_size", "bole_qk_norm_rotary",
           "bind_window_attention", "bole_window_attention", "bole_window_workspace_size",
           "bind_delta_commit_path", "bind_delta_prefill", "bind_delta_step",
           "bind_delta_tree_verify", "bole_delta_commit_path", "bole_delta_prefill",
           "bole_delta_prefill_workspace_size", "bole_delta_step", "bole_delta_tree_verify",
           "bind_build_tree", "bole_build_tree", "bind_tree_accept", "bole_tree_accept", "bind_commit_path", "bind_commit_path_layers", "bind_tree_verify",
           "bind_tree_verify_lazy_commit", "bind_tree_verify_lazy_commit_layers",
           "bind_tree_verify_layers", "bole_commit_path", "bole_commit_path_layers",
           "bole_tree_prepare", "bole_tree_verify", "bole_tree_verify_lazy_commit",
           "bole_tree_verify_lazy_commit_layers", "bole_tree_verify_layers",
           "bole_tree_verify_naive", "BoleError", "MAX_TREE_NODES"]
