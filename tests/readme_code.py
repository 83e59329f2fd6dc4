"""The README's Python lines."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def block():
    with open(os.path.join(ROOT, "README.md")) as f:
        return re.search(r"```python\n(.*?)```", f.read(), re.S).group(1)


def part(title):
    """The lines from the comment that starts with `title` to the next one."""
    text = block()
    start = text.index(f"# {title}")
    end = text.find("\n# ", start + 1)
    return text[start:] if end < 0 else text[start:end + 1]
