"""Lists of gradients whose tensors change between calls, on the GPU: a call takes the values that the tensors
hold then, and writes those alone.  (Sums of small whole numbers are exact here, and a factor that is a power of two.)"""

import threading

import pytest
import torch

import fp8_transformer_gb300 as te

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_resized_at_the_same_address():
    p = torch.full((1000,), 4.0, device=DEV)
    whole = p.data
    plan, norm = te.GradList([p]), torch.empty(1, device=DEV)
    te.te_grad_norm(plan, norm)
    assert abs(norm.item() - 16000 ** 0.5) <= 2.0 ** -19 * 16000 ** 0.5
    at = p.data_ptr()
    p.resize_(16)
    assert p.data_ptr() == at
    te.te_clip_grad_norm(plan, 8.0, norm, epsilon=0.0)  # 16 values of 4: a norm of 16, a factor of 1 / 2
    assert norm.item() == 16.0
    assert bool((whole[:16] == 2.0).all()) and bool((whole[16:] == 4.0).all())
    p.data = whole[:4]
    te.te_clip_grad_norm(plan, 1.0, norm, epsilon=0.0)  # 4 of 2: 4, a quarter
    assert norm.item() == 4.0
    assert bool((whole[:4] == 0.5).all()) and bool((whole[4:16] == 2.0).all()) and bool((whole[16:] == 4.0).all())


def test_another_type_at_the_same_address():
    p = torch.zeros(64, device=DEV)
    plan, norm = te.GradList([p]), torch.empty(1, device=DEV)
    te.te_grad_norm(plan, norm)
    p.data = p.data.view(torch.bfloat16)[:64]
    p.fill_(2.0)
    te.te_clip_grad_norm(plan, 4.0, norm, epsilon=0.0)
    assert norm.item() == 16.0 and bool((p == 0.5).all())


def test_an_out_that_no_longer_fits_is_refused():
    p, o = torch.ones(64, device=DEV), torch.zeros(64, device=DEV)
    plan, norm = te.GradList([p], [o]), torch.empty(1, device=DEV)
    te.te_clip_grad_norm(plan, 4.0, norm, epsilon=0.0)
    assert norm.item() == 8.0 and bool((o == 0.5).all())
    o.data = o.data[:10]
    with pytest.raises(ValueError):
        te.te_clip_grad_norm(plan, 4.0, norm)
    p.data = p.data[::2]
    with pytest.raises(ValueError):
        te.te_grad_norm(plan, norm)


def test_one_list_from_several_threads():
    ps = [torch.full((n,), 1.0, device=DEV) for n in (400, 41, 1, 2000)]
    plan, want = te.GradList(ps), float(torch.tensor(2442.0).sqrt())
    got, errors = [], []

    def work():
        try:
            norm = torch.empty(1, device=DEV)
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    te.te_grad_norm(plan, norm)
            torch.cuda.synchronize()
            got.append(norm.item())
        except Exception as e:  # pragma: no cover
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and len(got) == 4 and all(abs(g - want) <= 2.0 ** -19 * want for g in got)
