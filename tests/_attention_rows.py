"""Cache rows of a tests' Problem set from given fp64 rows, in either cache format."""
import torch

from tests import _attention as ref

BF = torch.bfloat16


def put(p, name, i, rows, first=0, scale=None):
    """Tokens first .. of request i get `rows` [n, Hkv, d] fp64 as their keys (name "k") or values ("v"); an e4m3 cache takes
    them quantised as kda_kv_write would, or as codes of the given scales [n, Hkv]."""
    at = first + torch.arange(len(rows))
    where = (p.table_cpu[i][at // p.page], slice(None), at % p.page)
    pages, exact = getattr(p, name), getattr(p, name + "d")
    if p.kind == BF:
        x = rows.to(BF)
        exact[where] = x.double()
        pages[where] = x.to(pages.device)
        return
    if scale is None:
        codes, scale = ref.quantise(rows)
    else:
        codes = ref.e4m3(rows / scale[..., None])
    exact[where] = codes * scale[..., None]
    pages.view(torch.uint8)[where] = codes.float().to(torch.float8_e4m3fn).view(torch.uint8).to(pages.device)
    getattr(p, name + "s")[where] = scale.float().to(pages.device)
