"""Paged-cache calls without a GPU: the descriptors' layout, the pure host
checks and the binding's refusals."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_descriptors_match_the_header(hd, tmp_path):
    structs = {"hd_paged_cache": hd.hd_paged_cache, "hd_paged_batch": hd.hd_paged_batch}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "hybrid_decode.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        s, f, v = line.split()
        assert int(v) == (ctypes.sizeof(structs[s]) if f == "size" else getattr(structs[s], f).offset), line


def descriptors(hd, **kw):
    """A good pair of descriptors with made-up addresses, changed by kw."""
    b = dict(block_table=4096, context=4096, token_offsets=4096, table_stride=8, max_blocks=8, batch=2, num_tokens=5,
             max_tokens=4, max_context=100)
    c = dict(k=4096, v=8192, page_stride=2 * 64 * 256, num_pages=10, page_size=64, k_scale=None, v_scale=None, bounds=None)
    for name, value in kw.items():
        (b if name in b else c)[name] = value
    return hd.hd_paged_batch(**b), hd.hd_paged_cache(**c)


def config(hd, **kw):
    return hd.Config(**dict(dict(layer_types=[0, 1], max_batch=4, max_context=1000), **kw))


@pytest.mark.parametrize("change,status", [
    ({}, 0), ({"block_table": None}, 1), ({"context": None}, 1), ({"batch": 0}, 1), ({"num_tokens": -1}, 1),
    ({"num_tokens": 0}, 0), ({"max_tokens": 0}, 1), ({"max_context": -1}, 1), ({"max_context": 0}, 0),
    ({"max_blocks": 0}, 1), ({"table_stride": 7}, 1), ({"table_stride": 90}, 0), ({"batch": 5}, 3),
    ({"max_context": 1001}, 3), ({"token_offsets": None}, 1),
    ({"token_offsets": None, "num_tokens": 2, "max_tokens": 1}, 0), ({"token_offsets": None, "num_tokens": 2, "max_tokens": 2}, 1),
    ({"k": None}, 1), ({"v": 8200}, 1), ({"bounds": 8}, 1), ({"num_pages": 0}, 1), ({"num_pages": 2 ** 31 - 1}, 1),
    ({"page_stride": 2 * 64 * 256 - 8}, 1), ({"page_stride": 2 * 64 * 256 + 4}, 1), ({"page_stride": 2 * 64 * 256 + 8}, 0),
    ({"page_size": 8}, 2), ({"page_size": 48}, 2), ({"page_size": 512}, 2), ({"page_size": 0}, 2), ({"page_size": 16}, 0),
    ({"k_scale": 16}, 1), ({"k_scale": 16, "v_scale": 16}, 1),
])
def test_host_check_of_bf16_descriptors(hd, change, status):
    assert hd.hd_validate_paged(config(hd), *descriptors(hd, **change)) == status


@pytest.mark.parametrize("change,status", [({}, 1), ({"k_scale": 16}, 1), ({"k_scale": 16, "v_scale": 16}, 0),
                                           ({"k_scale": 16, "v_scale": 16, "page_stride": 2 * 64 * 256 + 8}, 1),
                                           ({"k_scale": 16, "v_scale": 16, "page_stride": 2 * 64 * 256 + 16}, 0)])
def test_host_check_of_e4m3_descriptors(hd, change, status):
    assert hd.hd_validate_paged(config(hd, kv_dtype=hd.HD_KV_FP8_E4M3), *descriptors(hd, **change)) == status


def test_host_check_takes_the_configuration_first(hd):
    b, c = descriptors(hd)
    assert hd.hd_validate_paged(config(hd, head_dim=128, rotary_dim_sliding=128), b, c) == 2
    assert hd._lib.hd_validate_paged(None, ctypes.byref(b), ctypes.byref(c)) == 1
    assert hd._lib.hd_validate_paged(ctypes.byref(config(hd).to_c()), None, ctypes.byref(c)) == 1


def test_calls_refuse_a_null_context(hd):
    b, c = (ctypes.byref(x) for x in descriptors(hd))
    assert hd._lib.rope_append_paged(None, 0, b, 4096, 2048, 4096, 512, 4096, 512, 4096, c, None) == 1
    assert hd._lib.attn_paged(None, 0, b, 4096, c, None, None, 4096, 4096, None) == 1
    assert hd._lib.select_pages(None, 0, b, 4096, c, 4, 1, 1, 4096, None) == 1
    assert hd._lib.attn_selected_pages(None, 0, b, 4096, c, 4096, 4, None, None, 4096, 4096, None) == 1


def test_binding_refuses_host_tensors(hd):
    pages = torch.zeros(4, 2, 64, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hd.paged_cache(pages, pages)
    with pytest.raises(ValueError):
        hd.paged_cache(pages, pages[:2])
    with pytest.raises(ValueError):
        hd.paged_batch(torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        hd.paged_batch(torch.zeros(3, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_binding_refuses_pages_of_another_device(hd, monkeypatch):
    from types import SimpleNamespace
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ctx = SimpleNamespace(cfg=SimpleNamespace(num_kv_heads=2, kv_dtype=hd.HD_KV_BF16))
    b, c = descriptors(hd)
    there, here = torch.device("cuda", 1), torch.device("cuda", 0)

    def pair(batch_device, cache_device):
        cache = hd.PagedCache(c, (), (4, 2, 64, 256), cache_device)
        cache.fp8 = False
        return hd.PagedBatch(b, (), batch_device), cache

    hd._check_paged(ctx, *pair(here, here))
    for devices in ((there, there), (here, there), (there, here)):
        with pytest.raises(ValueError):
            hd._check_paged(ctx, *pair(*devices))


def test_binding_checks_rows(hd):
    one = torch.zeros(5, 2, 256, dtype=torch.bfloat16)[:, :1]          # one head of wider rows
    hd._check_rows("k", one, (5, 1, 256), torch.bfloat16, one.device, True)
    with pytest.raises(ValueError):
        hd._check_rows("k", one, (5, 1, 256), torch.bfloat16, one.device)
    for bad in (torch.zeros(5, 1, 512, dtype=torch.bfloat16)[..., ::2], one.float(), one[:4]):
        with pytest.raises(ValueError):
            hd._check_rows("k", bad, (5, 1, 256), torch.bfloat16, one.device, True)
