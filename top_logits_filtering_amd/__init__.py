"""MI355X-native top-k / top-p logits filter (libtopktopp) and its Python binding."""

from .binding import (  # noqa: F401
    EXPORTED_SYMBOLS,
    LIB_PATH,
    TopKTopPError,
    apply_top_k_top_p,
    apply_top_k_top_p_with_sorted,
    beam_backtrace,
    beam_reorder_states,
    beam_search_select,
    beam_search_select_workspace,
    cache_pages_compact,
    cache_pages_fork,
    cache_pages_resize,
    cache_pages_resize_workspace,
    last_error,
    load_library,
    sample_top_k_top_p,
    set_plan_policy,
    speculative_verify,
    speculative_verify_workspace,
    top_k_top_p_sorted_survivors,
)
