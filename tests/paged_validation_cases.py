"""Host-side argument checks of the paged-cache entry points, called with addresses that are
never dereferenced.  Every call here must return during host validation; the module is only
run in a child process that sees no GPU.  Run as a script it prints the return codes as JSON."""
import json
import sys

from speculative_decoding_tree_spec_gb300 import binding
from speculative_decoding_tree_spec_gb300.binding import NodeLayout, PagedLayout

FAKE = 1 << 20  # a 256-byte aligned address that the host never dereferences
CACHE = dict(n_pages=10, page_size=16, n_kv_heads=2, head_dim=64, page_stride=2048, pos_stride=128,
             head_stride=64)
NODES = dict(batch_stride=512, node_stride=256, head_stride=64)

APPEND = [
    (dict(B=0), 0),
    (dict(N=0), 0),
    (dict(dtype=5), -2),
    (dict(B=-1), -1),
    (dict(rot_dim=65), -1),
    (dict(rot_dim=-16), -1),
    (dict(rot_dim=24), -3),
    (dict(n_positions=-1), -1),
    (dict(flags=2), -1),
    (dict(k=None), -1),
    (dict(v=None), -1),
    (dict(q=None), -1),
    (dict(out_q=None), -1),
    (dict(k_cache=None), -1),
    (dict(v_cache=None), -1),
    (dict(page_table=None), -1),
    (dict(prefix_len=None), -1),
    (dict(cos_sin=None), -1),
    (dict(k=FAKE + 8), -3),
    (dict(v_cache=FAKE + 2), -3),
    (dict(k_layout=dict(NODES, node_stride=4)), -3),
    (dict(cache=dict(CACHE, pos_stride=130)), -3),
    (dict(cache=dict(CACHE, page_size=0)), -1),
    (dict(cache=dict(CACHE, n_kv_heads=0)), -1),
    (dict(cache=dict(CACHE, head_dim=60), rot_dim=32), -3),
    (dict(cache=dict(CACHE, head_dim=1040)), -6),
    (dict(cache=dict(CACHE, page_stride=-2048)), -1),
    (dict(max_pages=1 << 28), -6),
    (dict(max_pages=-1), -1),
    (dict(B=1 << 20, N=1 << 20), -6),
]

ATTEND = [
    (dict(B=0), 0),
    (dict(N=0), 0),
    (dict(dtype=2), -2),
    (dict(n_q_heads=3), -1),
    (dict(n_q_heads=0), -1),
    (dict(N=-1), -1),
    (dict(shared_len=-16), -1),
    (dict(shared_len=8), -1),
    (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1),
    (dict(q=None), -1),
    (dict(k_cache=None), -1),
    (dict(v_cache=None), -1),
    (dict(page_table=None), -1),
    (dict(prefix_len=None), -1),
    (dict(out=None), -1),
    (dict(workspace=None), -1),
    (dict(cache=dict(CACHE, head_dim=136)), -6),
    (dict(cache=dict(CACHE, head_dim=60)), -3),
    (dict(cache=dict(CACHE, head_stride=68)), -3),
    (dict(cache=dict(CACHE, page_size=-1)), -1),
    (dict(cache=dict(CACHE, n_pages=-1)), -1),
    (dict(q_layout=dict(NODES, head_stride=4)), -3),
    (dict(out_layout=dict(NODES, batch_stride=4)), -3),
    (dict(q=FAKE + 2), -3),
    (dict(out=FAKE + 8), -3),
    (dict(workspace=FAKE + 128), -4),
    (dict(ws_bytes=1000), -4),
    (dict(max_pages=1 << 28), -6),
    (dict(B=1 << 20, N=1 << 10), -6),
]

COMMIT = [
    (dict(B=0), 0),
    (dict(n_planes=0), 0),
    (dict(n_heads=0), 0),
    (dict(row_bytes=0), 0),
    (dict(B=-1), -1),
    (dict(W=0), -1),
    (dict(page_size=0), -1),
    (dict(n_pages=-1), -1),
    (dict(plane_stride=-16), -1),
    (dict(cache=None), -1),
    (dict(page_table=None), -1),
    (dict(prefix_len=None), -1),
    (dict(accepted_path=None), -1),
    (dict(accept_len=None), -1),
    (dict(cache=FAKE + 8), -3),
    (dict(row_bytes=24), -3),
    (dict(pos_stride=72), -3),
    (dict(head_stride=8), -3),
    (dict(row_bytes=128, pos_stride=64), -1),
    (dict(max_pages=1 << 30), -6),
    (dict(n_planes=1 << 20, n_heads=1 << 12), -6),
]


def _append(L, **kw):
    a = dict(q=FAKE, out_q=FAKE, k=FAKE, v=FAKE, dtype=1, B=2, N=2, n_q_heads=4, k_cache=FAKE,
             v_cache=FAKE, cache=CACHE, page_table=FAKE, max_pages=4, prefix_len=FAKE, counts=None,
             position_ids=None, cos_sin=FAKE, n_positions=100, rot_dim=64, flags=0, k_layout=NODES)
    a.update(kw)
    n = NodeLayout(**NODES)
    return L.spec_paged_append_rope(
        a["q"], n, a["out_q"], n, a["k"], NodeLayout(**a["k_layout"]), a["v"], n, a["dtype"], a["B"],
        a["N"], a["n_q_heads"], a["k_cache"], a["v_cache"], PagedLayout(**a["cache"]),
        a["page_table"], a["max_pages"], a["prefix_len"], a["counts"], a["position_ids"],
        a["cos_sin"], a["n_positions"], a["rot_dim"], a["flags"], None)


def _attend(L, **kw):
    a = dict(q=FAKE, q_layout=NODES, k_cache=FAKE, v_cache=FAKE, cache=CACHE, dtype=1, B=2, N=2,
             n_q_heads=4, page_table=FAKE, max_pages=4, prefix_len=FAKE, counts=None, mask=None,
             shared_len=0, scale=0.125, out=FAKE, out_layout=NODES, lse=None, workspace=FAKE,
             ws_bytes=1 << 40)
    a.update(kw)
    return L.spec_tree_attention_paged(
        a["q"], NodeLayout(**a["q_layout"]), a["k_cache"], a["v_cache"], PagedLayout(**a["cache"]),
        a["dtype"], a["B"], a["N"], a["n_q_heads"], a["page_table"], a["max_pages"],
        a["prefix_len"], a["counts"], a["mask"], a["shared_len"], a["scale"], a["out"],
        NodeLayout(**a["out_layout"]), a["lse"], a["workspace"], a["ws_bytes"], None)


def _commit(L, **kw):
    a = dict(cache=FAKE, B=2, n_planes=2, n_heads=2, n_pages=10, page_size=4, plane_stride=4096,
             page_stride=512, pos_stride=128, head_stride=64, row_bytes=64, page_table=FAKE,
             max_pages=4, prefix_len=FAKE, accepted_path=FAKE, accept_len=FAKE, W=3)
    a.update(kw)
    return L.spec_commit_accepted_path_paged(*a.values(), None)


def main():
    L = binding.lib()
    print(json.dumps({"append": [_append(L, **kw) for kw, _ in APPEND],
                      "attend": [_attend(L, **kw) for kw, _ in ATTEND],
                      "commit": [_commit(L, **kw) for kw, _ in COMMIT]}))


if __name__ == "__main__":
    sys.exit(main())
