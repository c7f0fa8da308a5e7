"""What the serving calls refuse and what they allow, and the workspaces that
they ask for."""
import ctypes

import pytest
import torch

import long_context_sparse_gb300 as dsa
from long_context_sparse_gb300 import build as dsa_build
from tests.test_serving import DEV, Case, check_case

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa._load()


def test_attention_refuses_what_overlaps(lib):
    """o, lse and the workspace may not meet what the call reads, or one
    another; q is the exception for o and lse, which are written behind it."""
    T, H, B, d, page = 8, 16, 4, 128, 64
    c = dsa.ServeConfig(n_pages=100, max_tokens=T, batch=B, max_blocks=10, page_size=page,
                        attn_heads=H, d_qk=d, d_v=d)
    r = ctypes.byref(c.c())
    nb = dsa.serve_workspace_size(c, dsa.SERVE_WS_PREFIX)
    size = dict(q=T * H * d * 2, k=100 * page * d * 2, v=100 * page * d * 2, prefix=16,
                table=B * 40, seq=B * 4, cu=B * 4 + 4, o=T * H * d * 2, lse=T * H * 4, ws=nb)
    at = {n: (i + 1) << 28 for i, n in enumerate(size)}
    assert max(size.values()) < 1 << 28

    def call(prefix_len=200, **over):
        a = {**at, **over}
        q, k, v, pt, table, seq, cu, o, lse, ws = (P(x) for x in a.values())
        return lib.dsa_prefix_attn(r, q, k, v, pt, prefix_len, table, seq, cu, o, lse, ws, nb,
                                   None)

    for w in ("o", "lse", "ws"):
        step = 256 if w == "ws" else 16
        for x in size:
            if x == w or (x == "q" and w != "ws"):
                continue
            assert call(**{w: at[x]}) == 1, (w, x)                                 # the same place
            assert call(**{w: at[x] + (size[x] - 1) // step * step}) == 1, (w, x)  # its end
            assert call(**{x: at[w] + (size[w] - 1) // 256 * 256}) == 1, (w, x)


def test_tables_and_append_refuse_a_workspace_in_their_buffers(lib):
    """The status word is latched while the kernels read and write: the header may
    not lie in anything of the call's, and anything may not end in it."""
    B, T, n_free, width, d, page = 4, 512, 100, 10, 128, 64
    c = dsa.ServeConfig(n_pages=100, max_tokens=T, batch=B, max_blocks=width, page_size=page,
                        d_qk=d, d_v=d)
    r, ws = ctypes.byref(c.c()), 1 << 40
    size = dict(cached=16, new=16, free=n_free * 4, table=B * width * 4, slots=T * 4, cu=20,
                seq=16, taken=4)
    at = {n: (i + 1) << 28 for i, n in enumerate(size)}

    def tables(ws, **over):
        a = [P(x) for x in {**at, **over}.values()]
        return lib.dsa_build_page_tables(r, *a[:3], n_free, *a[3:], P(ws), 256, None)

    for x in at:
        assert tables(at[x]) == 1, x
        assert tables(at[x] + (size[x] - 1) // 256 * 256) == 1, x
        assert tables(ws, **{x: ws + 240}) == 1, x
    cache = 100 * page * d * 2
    size2 = dict(slots=T * 4, k_new=T * d * 2, v_new=T * d * 2, k=cache, v=cache)
    at2 = {n: (i + 1) << 28 for i, n in enumerate(size2)}

    def append(ws, **over):
        a = [P(x) for x in {**at2, **over}.values()]
        return lib.dsa_append_cache(r, *a, P(ws), 256, None)

    for x in at2:
        assert append(at2[x]) == 1, x
        assert append(at2[x] + (size2[x] - 1) // 256 * 256) == 1, x
        assert append(ws, **{x: ws + 240}) == 1, x


@pytest.mark.parametrize("T,H", [(1, 16), (64, 16), (64, 128), (1000, 64)])
def test_workspace_of_a_batch_that_is_mostly_idle(lib, T, H):
    """A request has partial results only with rows of its own, so requests beyond
    the query tokens add their place in the plan (12 bytes) and no more."""
    size = lambda B: dsa.serve_workspace_size(
        dsa.ServeConfig(n_pages=100, max_tokens=T, batch=B, max_blocks=10, attn_heads=H),
        dsa.SERVE_WS_PREFIX)
    assert size(65536) - size(T) <= 12 * 65536 + 256
    # of the rows: two lists of keys a row block, a request each, a part a pair
    slot = 128 * (4 * 512 + 16)
    assert size(T) <= 512 + 12 * (T + 1) + 256 + (2 * (-(-T * H // 128)) + T + 80) * slot


def test_a_scale_that_overflows_in_base_two_is_refused(lib):
    """The weights are powers of 2 of scale * log2(e) times a difference of scores,
    0 of them for the largest: 0 * inf would make every row NaN."""
    size = lambda s: dsa.serve_workspace_size(
        dsa.ServeConfig(n_pages=10, max_tokens=1, batch=1, max_blocks=1, sm_scale=s),
        dsa.SERVE_WS_PREFIX)
    for s in (2.4e38, 3.4e38):
        with pytest.raises(dsa.DsaError) as e:
            size(s)
        assert e.value.code == 1
    assert size(2.3e38) == size(0.0)


@pytest.mark.gpu
def test_outputs_over_the_queries_and_an_empty_prefix_table():
    """o in q's place; and, behind no prefix, a prefix table that lies anywhere (it
    is not read)."""
    for prefix in (0, 700):
        c = Case([1, 3, 20], [40, 300, 20], prefix, 16, 256, 64, 1, seed=prefix)
        ref = c.run()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        q, lse = c.q.to(DEV), torch.zeros(ref[1].shape, device=DEV)
        ws = dsa.serve_workspace(c.cfg, dsa.SERVE_WS_PREFIX, DEV)
        table = c.prefix_table.to(DEV) if prefix else lse.view(torch.int32).view(-1)
        dsa.prefix_attn(c.cfg, q, c.k.to(DEV), table, prefix, c.table.to(DEV), i32(c.seq),
                        i32(c.cu), o=q, lse=lse, ws=ws)
        assert dsa.get_device_status(ws) == 0
        assert torch.equal(q.cpu(), ref[0]) and torch.equal(lse.cpu(), ref[1])


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,prefix", [(1, 16, 0), (7, 16, 300), (40, 128, 3000)])
def test_nothing_is_written_past_the_workspace(T, H, prefix):
    """More requests than query tokens, one token for each of T of them: the most
    units that T tokens make."""
    B = 300
    new = [0] * B
    for b in range(T):
        new[7 * b] = 1
    c = Case(new, [n + b % 90 for b, n in enumerate(new)], prefix, H, 512, 64, 1, seed=T)
    need = dsa.serve_workspace_size(c.cfg, dsa.SERVE_WS_PREFIX)
    ws = torch.zeros(need + (1 << 20), dtype=torch.uint8, device=DEV)
    ws[need:] = 77
    check_case(c, ws=ws)
    assert (ws[need:] == 77).all()
