"""FP64 CPU oracle (test infrastructure only; see kvgqa_oracle.py and, for the
paged cache, paged_oracle.py)."""
from .kvgqa_oracle import *  # noqa: F401,F403
from .paged_oracle import *  # noqa: F401,F403
from . import kvgqa_oracle, paged_oracle  # noqa: F401
