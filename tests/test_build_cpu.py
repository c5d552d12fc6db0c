"""CPU tests of the build: of the compiler's output only the lines about the features that the build itself turns off are
dropped."""
import sys

from kda_gated_delta_chunk_amd import build


def said(*lines):
    return build._run([sys.executable, "-c", "print(%r)" % "\n".join(lines)]).splitlines()


def test_only_known_features_are_silent():
    known = ["'%s' is not a recognized feature for this target (ignoring feature)" % f for f in build.FEATURES]
    other = ["'-dot13-inst' is not a recognized feature for this target (ignoring feature)", "warning: a register spills"]
    assert said(known[0], other[0], known[1], other[1]) == other


def test_the_features_are_those_of_the_flags():
    given = build.FLAGS + [f for more in build.FILE_FLAGS.values() for f in more]
    off = {b for a, b in zip(given, given[1:]) if a == "-Xclang" and b.startswith("-") and b != "-target-feature"}
    assert off == set(build.FEATURES)
