"""csrc/choices.hpp asked which kernels an attention call takes on 256 CUs."""
from host_program import compile_choices

CUS = 256
_CALL = "fp4::AttentionCall{(int)dim, e4m3 != 0, T, batch, (int)q_heads, (int)heads, room, (int)window, (int)sinks, %s}"


def prompt_choice(directory):
    """dim, e4m3, T, batch, query heads, heads, room, window, sinks -> waves, splits, heads of a join's workgroup (0: no join)."""
    return compile_choices(directory, f"""
  long long dim, e4m3, T, batch, q_heads, heads, room, window, sinks;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld", &dim, &e4m3, &T, &batch, &q_heads, &heads, &room, &window, &sinks) == 9) {{
    const auto w = fp4::prompt_way({_CALL % "false"}, {CUS});
    std::printf("%d %d %d\\n", w.waves, w.splits, w.wide);
  }}""")


def decode_choice(directory):
    """dim, e4m3, batch, query heads, heads, room, window, sinks, heads side by side -> heads of a workgroup, whole, pieces, heads of a
    join's workgroup (0: no join)."""
    return compile_choices(directory, f"""
  long long dim, e4m3, batch, q_heads, heads, room, window, sinks, beside;
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld", &dim, &e4m3, &batch, &q_heads, &heads, &room, &window, &sinks, &beside) == 9) {{
    const long long T = batch;
    const auto w = fp4::decode_way({_CALL % "beside != 0"}, {CUS});
    std::printf("%d %d %lld %d\\n", w.beside, w.whole, (long long)w.most, w.wide);
  }}""")
