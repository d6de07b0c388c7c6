// The persistent kernels' scheduler (stream_common.cuh) on the host: schedulers as threads that take
// turns, a unit each, in one fixed order.
#include <condition_variable>
#include <mutex>
#include <thread>
#include <vector>

#include "stream_common.cuh"

using namespace moe;

namespace {
// Lets one of the threads run at a time, round robin over those that have not ended.
class Turns {
 public:
  explicit Turns(int n) : live_(n, true) {}
  void wait(int i) {
    std::unique_lock<std::mutex> l(m_);
    c_.wait(l, [&] { return now_ == i; });
  }
  void pass(int i, bool end) {
    std::lock_guard<std::mutex> l(m_);
    if (end) live_[i] = false;
    const int n = (int)live_.size();
    for (int j = 1; j <= n; ++j) {
      now_ = (i + j) % n;
      if (live_[now_]) break;
    }
    c_.notify_all();
  }

 private:
  std::mutex m_;
  std::condition_variable c_;
  std::vector<bool> live_;
  int now_ = 0;
};
}  // namespace

// n schedulers over E experts (counts[e] rows each) and a shared one.  The first n_first run, in turns;
// the others start when those have ended.  Published units go to out, 8 ints each: scheduler, kind,
// group, weight tile, first token, rows, first row, token tile's number.  Returns their number (of the
// first n_first schedulers: *from_first).
extern "C" int run_schedulers(const int *counts, int E, int n_shared, int T, int k, int bt,
                              int up_tiles, int down_tiles, int n, int n_first, int by_position,
                              int *out, int max_units, int *from_first) {
  StreamBase p{};
  p.E = E;
  p.n_shared = n_shared;
  p.T = T;
  p.k = k;
  std::vector<int> mem((StreamTables::BYTES + 3) / 4);
  const StreamTables tb(mem.data(), E, n_shared);
  tb.offsets[0] = 0;
  for (int e = 0; e < E; ++e) tb.offsets[e + 1] = tb.offsets[e] + counts[e];
  tb.tile_prefix[0] = 0;
  for (int o = 0; o < E + n_shared; ++o)
    tb.tile_prefix[o + 1] =
        tb.tile_prefix[o] + (group_rows(p, tb, group_at(p, o)) + bt - 1) / bt;

  int counter = 0, units = 0;
  auto run = [&](int begin, int end) {
    Turns turns(end - begin);
    std::vector<std::thread> threads;
    for (int me = begin; me < end; ++me)
      threads.emplace_back([&, me] {
        const int i = me - begin;
        turns.wait(i);
        auto claim = [&] { return counter++; };
        const Tickets first = by_position ? tickets_by_position(me, n) : tickets_claimed(claim(), claim);
        schedule_units(p, tb, bt, up_tiles, down_tiles, first, claim, [&](const Unit &r) {
          if (r.kind < 0) return true;
          if (units == max_units) return false;
          const int row[8] = {me, r.kind, r.g, r.mt, r.tok0, r.n, r.row0, r.tile};
          for (int j = 0; j < 8; ++j) out[units * 8 + j] = row[j];
          ++units;
          turns.pass(i, false);
          turns.wait(i);
          return true;
        });
        turns.pass(i, true);
      });
    for (auto &t : threads) t.join();
  };
  run(0, n_first);
  *from_first = units;
  run(n_first, n);
  return units;
}
