"""A star import of the package has every call of the header and every public name."""
import combine_moe_layout_05_gb300 as moe
from combine_moe_layout_05_gb300 import _binding


def test_star_import_has_every_call():
    scope = {}
    exec("from combine_moe_layout_05_gb300 import *", scope)
    for name in moe.declared_functions():
        assert scope.get(name) is getattr(_binding, name), name
    public = {n for n, v in vars(moe).items() if getattr(v, "__module__", None) == _binding.__name__}
    assert public <= set(moe.__all__) and len(set(moe.__all__)) == len(moe.__all__)
