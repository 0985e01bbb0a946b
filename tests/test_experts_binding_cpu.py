"""The package's public names: what `from combine_moe_layout_02_amd import *` gives. Needs no GPU."""

import combine_moe_layout_02_amd as moe


def test_every_public_name_is_exported():
    """Each call of the C ABI that has a binding of its name, the tuples that calls return or take, and the
    constants that are arguments or results."""
    names = {n for n in moe.EXPORTED if hasattr(moe, n)}
    names |= {n for n in vars(moe) if n.startswith("MOE_")}
    names |= {n for n, v in vars(moe).items() if isinstance(v, type) and issubclass(v, tuple) and v.__module__ == moe.__name__}
    assert len(names) > 40
    missing = sorted(names - set(moe.__all__))
    assert not missing, missing
    assert len(set(moe.__all__)) == len(moe.__all__) and all(hasattr(moe, n) for n in moe.__all__)
