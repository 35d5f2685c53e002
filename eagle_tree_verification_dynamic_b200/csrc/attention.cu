// Host plan of the tree attention ("Tree Attention" verification of the EAGLE
// notes, "3.Verify"): how many CTAs share the tile list, and the workspace that
// holds the partials of units cut by CTA range boundaries.  The kernels are in
// attention_tc.cu.
#include <atomic>

#include "eagle_internal.h"

namespace eagle {

namespace {
std::atomic<unsigned long long> g_probe_ns{0};
}  // namespace

unsigned long long attention_wait_probe_ns() { return g_probe_ns.load(std::memory_order_relaxed); }

namespace {
int groups(const AttnShape& a, int nodes) { return (nodes * (a.Hq / a.Hkv) + a.unit_rows() - 1) / a.unit_rows(); }
}  // namespace

int attention_row_groups(const AttnShape& a) { return groups(a, a.n); }

int attention_shared_row_groups(const AttnShape& a) {
  return a.Lshared > 0 ? groups(a, a.B * a.n) : 0;
}

int attention_ctas(const AttnShape& a) {
  long long span = a.Lmax;
  if (a.window > 0) {  // the window's keys and the sinks before them
    const long long seen = (long long)a.window + a.sinks;
    if (seen < span) span = seen;
  }
  const auto tiles = [](long long keys) { return (keys + kAttnKeysPerTile - 1) / kAttnKeysPerTile; };
  const long long T_max =
      (long long)a.B * a.Hkv * attention_row_groups(a) * (tiles(span) + tiles(a.n)) +
      (long long)a.Hkv * attention_shared_row_groups(a) * tiles(a.Lshared);
  const int sms = device_sm_count();
  return (int)(T_max < sms ? T_max : sms);
}

AttnWorkspace attention_ws_layout(const AttnShape& a) {
  AttnWorkspace w;
  const int C = attention_ctas(a);
  const size_t U = (size_t)a.B * a.Hkv * attention_row_groups(a) +
                   (size_t)a.Hkv * attention_shared_row_groups(a);
  const size_t slots = (size_t)C + U;
  w.status_off = 0;
  w.cta_status_off = 256;
  w.part_lse_off = align_up(w.cta_status_off + sizeof(int) * (size_t)C, 256);
  w.part_o_off = align_up(w.part_lse_off + sizeof(float) * slots * a.unit_rows(), 256);
  w.bytes = align_up(w.part_o_off + sizeof(float) * slots * a.unit_rows() * (size_t)a.D, 256);
  return w;
}

}  // namespace eagle

extern "C" EAGLE_API void eagle_debug_attention_wait_probe(unsigned long long limit_ns) {
  eagle::g_probe_ns.store(limit_ns, std::memory_order_relaxed);
}
