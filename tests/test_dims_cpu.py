"""The record of a Dims that the calls of the 8-bit cache read by its address."""
import copy
import ctypes
import dataclasses
import pickle
import threading

import sliding_window_gqa_chunk_b200 as swa


def test_threads_that_ask_first_together_get_one_record(monkeypatch):
    """Two threads, each held inside the making of the record until the other is there too: the address that either
    got is that of the record that the Dims keeps."""
    d = swa.Dims(1, 2, 1, 16, 64, 0.25)
    both, made = threading.Barrier(2, timeout=10), []
    plain = swa.Dims.c

    def slow(self):
        record = plain(self)
        both.wait()
        return record

    monkeypatch.setattr(swa.Dims, "c", slow)

    def ask():
        made.append(d._dims_addr)

    threads = [threading.Thread(target=ask) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    monkeypatch.undo()
    assert made == [ctypes.addressof(d._record)] * 2 == [d._dims_addr] * 2


@dataclasses.dataclass(frozen=True)
class Layer(swa.Dims):
    name: str = "?"


def test_copies_of_a_kind_of_dims_stay_of_their_kind():
    a = Layer(1, 2, 1, 16, 64, 0.25, "bf16", "first")
    object.__setattr__(a, "note", [1])
    address = a._dims_addr
    for b in (copy.copy(a), copy.deepcopy(a), pickle.loads(pickle.dumps(a))):
        assert type(b) is Layer and b == a and b.note == [1]
        assert b._dims_addr != address and b._record.batch == 1
