"""A comparison that a NaN on either side fails."""


def within(got, ref, bound):
    """Whether every |got - ref| is a number and at most its bound."""
    return bool(((got.double() - ref).abs() <= bound).all())
