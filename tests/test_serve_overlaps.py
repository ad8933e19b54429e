"""No array that an attention-layer call writes may overlap another of its arrays: every pair, on the host
(no GPU needed: the addresses are never dereferenced)."""
import ctypes

import pytest

from gated_deltanet_rule_gb300 import build as gbuild
from gated_deltanet_rule_gb300 import gdr

# each call: (arguments in order, the arrays among them; written ones). Sizes: B = 2 (rows 8), N = 3, heads 4 / 2 of 128
B, N, HQ, HK, D, R, P, PAGE, M, F, V = 2, 3, 4, 2, 128, 64, 9, 16, 4, 2, 100
BIG = 1 << 34

CALLS = {
    "gdr_qk_norm_rope": ("q k q_w k_w inv_freq pos".split() + [1e-6, 0] + "q_out k_out".split()
                         + [B, N, HQ, HK, D, R, 512, 128, 256, 128, 1, None], "q_out k_out"),
    "gdr_qk_norm_rope_append": ("q k v q_w k_w inv_freq pos".split() + [1e-6, 0] + "q_out k_pages v_pages table ctx lengths".split()
                                + [P, PAGE, M, B, N, HQ, HK, D, R, 512, 128, 256, 128, 256, 128, 1, None], "q_out k_pages v_pages"),
    "gdr_qk_norm_rope_backward": ("q k q_w k_w inv_freq pos dq_out dk_out".split() + [1e-6, 0] + "dq dk dq_w dk_w".split()
                                  + [B, N, HQ, HK, D, R, 512, 128, 256, 128, 1, "ws", BIG, None], "dq dk dq_w dk_w ws"),
    "gdr_tree_attn": ("q k_pages v_pages table ctx lengths mask".split() + [0.1] + "o lse".split()
                      + [B, N, HQ, HK, D, P, PAGE, M, 1, "ws", BIG, None], "o lse ws"),
    "gdr_verify_draft": ("tokens parents lengths p q u u_next path n_path next_token".split() + [B, N, V, 0, None],
                         "path n_path next_token"),
    "gdr_cache_reserve": ("table ctx refs rows".split() + [3, F, 8, M, P, PAGE, "ws", BIG, None], "table refs ws"),
    "gdr_cache_fork": ("k_cache v_cache table ctx refs src dst".split() + [F, 8, M, 2, P, PAGE, 512, "ws", BIG, None],
                       "k_cache v_cache table ctx refs ws"),
    "gdr_cache_free": ("table ctx refs rows".split() + [F, 8, M, P, None], "table ctx refs"),
    "gdr_cache_compact": ("k_cache v_cache table ctx path n_path new_ctx".split() + [B, 5, M, 2, P, PAGE, 512, None],
                          "k_cache v_cache new_ctx"),
}


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdr.lib()


@pytest.mark.parametrize("name", CALLS)
def test_every_written_array_keeps_apart(L, name):
    args, written = CALLS[name]
    arrays = [a for a in args if isinstance(a, str)]
    for out in written.split():
        for other in arrays:
            if other == out:
                continue
            at = {a: ctypes.c_void_p((n + 1) << 40) for n, a in enumerate(arrays)}
            at[out] = at[other]
            st = getattr(L, name)(*[at[a] if isinstance(a, str) else a for a in args])
            assert st == gdr.GDR_ERR_INVALID_ARG and "overlaps" in L.gdr_last_error_message().decode(), (out, other)
