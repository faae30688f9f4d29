"""Memory that an attention call writes and shares with something else is refused before any launch (no GPU needed)."""
import ctypes
import re

import pytest

import gated_delta_rule_37_gb300 as gdr
from tests.test_abi_attn import BF16, INVALID, UNSUPPORTED, P, _append, _fwd, _step, lib  # noqa: F401

# 4 tokens of 8 query heads and 2 key heads of 64, bf16: rows of 1024 and 256 bytes; caches of 9 pages of 16: 36864
M = 1 << 20
APPEND = dict(q=P(M), ldq=512, k=P(2 * M), ldk=128, v=P(3 * M), ldv=128, qo=P(4 * M), ldqo=512, ko=P(5 * M), ldko=128,
              kc=P(6 * M), vc=P(7 * M))
FWD = dict(q=P(M), k=P(2 * M), v=P(3 * M), o=P(4 * M))
STEP = dict(q=P(M), kc=P(2 * M), vc=P(3 * M), o=P(4 * M), ws=P(5 * M))


def _message(lib):
    return lib.gdr_last_error().decode()


@pytest.mark.parametrize("kw,names", [
    (dict(vc=P(6 * M)), "k_cache is written and overlaps v_cache"),
    (dict(vc=P(6 * M + 36864 - 16)), "k_cache is written and overlaps v_cache"),
    (dict(qo=P(M + 16)), "q_out is written and overlaps q"),           # in place, but not quite
    (dict(qo=P(2 * M - 16)), "q_out is written and overlaps k"),
    (dict(ko=P(M + 3 * 1024 + 1008)), "k_out is written and overlaps q"),
    (dict(ko=P(3 * M)), "k_out is written and overlaps v"),
    (dict(ko=P(4 * M)), "q_out is written and overlaps k_out"),
    (dict(kc=P(2 * M - 36864 + 16)), "k_cache is written and overlaps k"),
    (dict(vc=P(5 * M - 16)), "k_out is written and overlaps v_cache"),
    # column blocks of one buffer of 12 heads, a block that begins a head too early
    (dict(q=P(M), ldq=768, qo=P(M), ldqo=768, k=P(M + 896), ldk=768, ko=P(M + 896), ldko=768), "q_out .* k"),
    (dict(q=P(M), ldq=768, qo=P(M), ldqo=768, k=P(M + 1024), ldk=768, ko=P(M + 1408), ldko=768), "q_out .* k_out"),
])
def test_append_refuses_shared_memory(lib, kw, names):
    assert _append(lib, **{**APPEND, **kw}) == INVALID
    assert re.search(names, _message(lib))


@pytest.mark.parametrize("o,name", [(M + 2048, "q"), (M - 4096 + 16, "q"), (2 * M + 512, "k"), (3 * M + 1008, "v"),
                                    (3 * M - 4080, "v")])
def test_fwd_refuses_shared_memory(lib, o, name):
    assert _fwd(lib, **{**FWD, "o": P(o)}) == INVALID
    assert _message(lib) == f"o is written and overlaps {name}"


@pytest.mark.parametrize("kw,names", [
    (dict(o=P(M + 16)), "o is written and overlaps q"),
    (dict(o=P(2 * M + 36864 - 16)), "o is written and overlaps k_cache"),
    (dict(o=P(3 * M + 16)), "o is written and overlaps v_cache"),
    (dict(ws=P(4 * M + 1024)), "workspace is written and overlaps o"),
    (dict(ws=P(M)), "workspace is written and overlaps q"),
    (dict(ws=P(2 * M + 256)), "workspace is written and overlaps"),
])
def test_step_refuses_shared_memory(lib, kw, names):
    assert _step(lib, **{**STEP, **kw}) == INVALID
    assert names in _message(lib)


def test_more_places_than_a_call_looks_at(lib):
    assert _fwd(lib, N=65535, Hkv=512, Hq=512) == UNSUPPORTED
    assert "2^24" in _message(lib)
    out = ctypes.c_size_t(0)
    assert lib.gdr_attn_step_workspace_size(65535, 65535, 512, 512, 64, 0, BF16, ctypes.byref(out)) == UNSUPPORTED
    assert lib.gdr_attn_step_workspace_size(65535, 65535, 256, 256, 64, 0, gdr.GDR_F32, ctypes.byref(out)) == 0
