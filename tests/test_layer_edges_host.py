"""Host-side checks of the layer norm's test helpers that need no GPU."""
import pytest

from test_train_host import AT, nsp, refused  # noqa: F401


def probe(nsp, back=False, fed=4, tries=10, **kw):
    v = dict(x=AT, x_row=8, weight=AT, bias=None, doc=None, N=6, D=8, dtype=nsp.NS_BF16,
             weight_dtype=nsp.NS_F32, eps=1e-5)
    call = dict(mean=AT, rstd=AT, dy=AT, dy_row=8, dx=AT, dweight=AT, dbias=AT, workspace=AT)
    if not back:
        call = dict(y=AT, mean=None, rstd=None)
    for k, x in kw.items():
        (v if k in v else call)[k] = x
    s = nsp._lib.ns_norm_inputs(*v.values())
    f = nsp._lib.ns_norm_probe_backward if back else nsp._lib.ns_norm_probe_forward
    return lambda: f(s, fed, tries, *call.values(), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw", [dict(fed=1), dict(fed=5), dict(x=None), dict(x_row=7), dict(dtype=5)])
def test_norm_probe_refuses(nsp, kw, back):
    refused(nsp, probe(nsp, back=back, **kw))


def test_norm_probe_of_nothing_is_ok(nsp):
    probe(nsp, N=0, x=None, y=None)()
